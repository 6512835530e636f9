"""Refusals of the operators around a recurrence (short convolution,
state-space scan, norms), through the C ABI and through the binding, and the
oracle's own pins. No GPU: everything here is refused before device work, or
there is nothing to do."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from gated_delta_rule_109_amd import kda
from oracle import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, BAD, UNSUP, WS = kda.KDA_OK, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
INT_MAX = 2 ** 31 - 1


def at(i, off=0):
    """Addresses 16 GiB apart that are never read."""
    return ctypes.c_void_p((i << 34) + 4096 + off)


def call(fn, defaults, given):
    assert set(given) <= set(defaults)
    return getattr(kda.lib(), fn)(*{**defaults, **given}.values())


def conv(**k):
    return call("kda_conv_prefill", dict(
        x=at(1), x_stride=64, weight=at(2), bias=at(3), dtype=0, cu=at(4), num_seqs=2, T=40, C=64, width=4, act=1,
        initial=at(5), final=at(6), y=at(7), stream=None), k)


def conv_step(**k):
    return call("kda_conv_step", dict(x=at(1), x_stride=64, weight=at(2), bias=at(3), dtype=0, state=at(5), N=3, C=64,
                                      width=4, act=1, y=at(7), stream=None), k)


def ssm(**k):
    return call("kda_ssm_prefill", dict(
        x=at(1), x_stride=4 * 64, dt=at(2), a=at(3), b=at(4), b_stride=64, c=at(5), c_stride=64, skip=at(6),
        dt_bias=at(7), softplus=1, dtype=0, cu=at(8), num_seqs=2, T=1000, H=4, G=2, N=32, P=64, initial=at(9),
        final=at(10), y=at(11), workspace=at(12), workspace_bytes=1 << 32, stream=None), k)


def ssm_step(**k):
    return call("kda_ssm_step", dict(
        x=at(1), x_stride=4 * 64, dt=at(2), a=at(3), b=at(4), b_stride=64, c=at(5), c_stride=64, skip=at(6),
        dt_bias=at(7), softplus=1, dtype=0, state=at(9), num_seqs=5, H=4, G=2, N=32, P=64, y=at(11), stream=None), k)


def gated(**k):
    return call("kda_gated_norm", dict(
        x=at(1), x_stride=4 * 64, gate=at(2), gate_stride=4 * 64, weight=at(3), per_head=0, dtype=0, T=7, H=4, D=64,
        act=2, gate_first=0, eps=1e-6, y=at(4), stream=None), k)


def residual(**k):
    return call("kda_residual_norm", dict(
        x=at(1), residual=at(2), gate=at(3), weight=at(4), post=at(5), scale=at(6), dtype=0, T=7, C=64, act=2,
        alpha=1.0, eps=1e-6, out=at(7), y=at(8), stream=None), k)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), UNSUP), (dict(C=0), BAD), (dict(C=kda.INT32_MAX, x_stride=1 << 40), BAD), (dict(width=1), BAD),
    (dict(width=5), BAD), (dict(act=2), BAD), (dict(act=-1), BAD), (dict(x_stride=63), BAD), (dict(x_stride=-64), BAD),
    (dict(x_stride=2 ** 62), BAD), (dict(weight=None), BAD), (dict(x=None), BAD), (dict(y=None), BAD),
    (dict(x=at(1, 2)), BAD), (dict(weight=at(2, 4)), BAD), (dict(bias=at(3, 8)), BAD), (dict(y=at(7, 2)), BAD),
    (dict(y=at(1)), BAD), (dict(y=at(2, 16)), BAD), (dict(y=at(3, 0)), BAD),
])
def test_both_convolutions_refuse(bad, status):
    assert conv(**bad) == status
    assert conv_step(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), BAD), (dict(T=(1 << 30) + 1), BAD), (dict(num_seqs=-1), BAD), (dict(cu=None), BAD),
    (dict(cu=at(4, 2)), BAD), (dict(initial=at(5, 4)), BAD), (dict(final=at(6, 4)), BAD), (dict(final=at(5, 16)), BAD),
    (dict(final=at(1)), BAD), (dict(y=at(5)), BAD), (dict(y=at(4)), BAD), (dict(final=at(7, 64)), BAD),
    (dict(num_seqs=1 << 25), BAD), (dict(num_seqs=0, T=0, x=None, y=None, initial=None), OK),
])
def test_conv_prefill_refuses(bad, status):
    assert conv(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(N=-1), BAD), (dict(N=(1 << 30) + 1), BAD), (dict(state=None), BAD), (dict(state=at(5, 4)), BAD), (dict(state=at(1)), BAD),
    (dict(y=at(5)), BAD), (dict(N=0, x=None, y=None, state=None), OK),
])
def test_conv_step_refuses(bad, status):
    assert conv_step(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=-1), UNSUP), (dict(N=48), UNSUP), (dict(N=512, b_stride=1024, c_stride=1024), UNSUP), (dict(P=8), UNSUP),
    (dict(P=24), UNSUP), (dict(P=272), UNSUP), (dict(H=0), BAD), (dict(G=0), BAD), (dict(G=3), BAD),
    (dict(softplus=2), BAD), (dict(x_stride=255), BAD), (dict(x_stride=260), BAD), (dict(b_stride=56), BAD),
    (dict(x_stride=(1 << 23) + 8), BAD), (dict(c_stride=68), BAD), (dict(b_stride=-64), BAD), (dict(x=None), BAD), (dict(dt=None), BAD), (dict(a=None), BAD),
    (dict(b=None), BAD), (dict(c=None), BAD), (dict(y=None), BAD), (dict(x=at(1, 8)), BAD), (dict(dt=at(2, 4)), BAD),
    (dict(b=at(4, 2)), BAD), (dict(skip=at(6, 4)), BAD), (dict(y=at(1)), BAD), (dict(y=at(2)), BAD), (dict(y=at(9)), BAD),
    (dict(y=at(4, 64)), BAD), (dict(H=1 << 20, x_stride=1 << 26, G=1, b_stride=32, c_stride=32, num_seqs=1 << 12), BAD),
])
def test_both_scans_refuse(bad, status):
    assert ssm(**bad) == status
    assert ssm_step(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), BAD), (dict(num_seqs=-1), BAD), (dict(cu=None), BAD), (dict(cu=at(8, 1)), BAD),
    (dict(initial=at(9, 4)), BAD), (dict(final=at(9, 64)), BAD), (dict(final=at(11)), BAD), (dict(workspace=None), WS),
    (dict(workspace=at(12, 16)), WS), (dict(workspace_bytes=1000), WS), (dict(workspace=at(9, 0)), BAD),
    (dict(workspace=at(1, 0)), BAD), (dict(T=1 << 28, H=16, x_stride=1024), BAD),
    (dict(T=0, num_seqs=0, x=None, dt=None, b=None, c=None, y=None, workspace=None), OK),
])
def test_ssm_prefill_refuses(bad, status):
    assert ssm(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(num_seqs=-1), BAD), (dict(state=None), BAD), (dict(state=at(9, 8)), BAD), (dict(state=at(1)), BAD),
    (dict(num_seqs=1 << 24, H=2, G=1), BAD),
    (dict(num_seqs=0, x=None, dt=None, b=None, c=None, y=None, state=None), OK),
])
def test_ssm_step_refuses(bad, status):
    assert ssm_step(**bad) == status


def test_ssm_workspace_covers_smaller_calls():
    size = kda.lib().kda_ssm_workspace_size
    assert size(1, 100, 32, 128, 128) == 0                   # one segment
    assert size(-1, 8192, 4, 64, 64) == 0 and size(1, 8192, 4, 48, 64) == 0 and size(1, 8192, 4, 64, 60) == 0
    for N in kda.SSM_STATES:
        for T in (64, 200, 1000, 8192, 100000):
            for H in (1, 2, 3, 7, 32, 100):
                for P in (16, 48, 64, 128, 256):
                    w = size(1, T, H, N, P)
                    for T2, H2, P2 in ((T * 2, H, P), (T, H + 1, P), (T, H, min(P + 16, 256)), (T + 1, H + 2, P)):
                        assert size(1, T2, H2, N, P2) >= w
                    assert size(9, T, H, N, P) >= w


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), UNSUP), (dict(T=-1), BAD), (dict(H=0), BAD), (dict(D=0), BAD),
    (dict(D=kda.NORM_MAX + 1, x_stride=1 << 20, gate_stride=1 << 20), BAD), (dict(T=1 << 29, H=4), BAD),
    (dict(act=3), BAD), (dict(act=-1), BAD), (dict(per_head=2), BAD), (dict(gate_first=-1), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=NAN), BAD), (dict(eps=INF), BAD), (dict(x_stride=255), BAD), (dict(gate_stride=0), BAD), (dict(x=None), BAD),
    (dict(weight=None), BAD), (dict(y=None), BAD), (dict(x=at(1, 2)), BAD), (dict(gate=at(2, 8)), BAD),
    (dict(weight=at(3, 4)), BAD), (dict(y=at(1)), BAD), (dict(y=at(2, 32)), BAD), (dict(y=at(3)), BAD),
    (dict(T=1 << 22, H=1, D=16384, x_stride=16384, gate_stride=16384, per_head=1, weight=at(1 << 8), gate=at(1 << 9),
          y=at(1 << 10)), BAD),                            # 2^32 threads
    (dict(T=0, x=None, y=None), OK),
])
def test_gated_norm_refuses(bad, status):
    assert gated(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), UNSUP), (dict(T=-1), BAD), (dict(C=0), BAD), (dict(C=kda.NORM_MAX + 1), BAD), (dict(act=3), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=NAN), BAD), (dict(alpha=NAN), BAD), (dict(alpha=-INF), BAD), (dict(x=None), BAD),
    (dict(weight=None), BAD), (dict(y=None), BAD), (dict(x=at(1, 4)), BAD), (dict(residual=at(2, 4)), BAD),
    (dict(gate=at(3, 4)), BAD), (dict(post=at(5, 4)), BAD), (dict(scale=at(6, 4)), BAD), (dict(out=at(7, 4)), BAD),
    (dict(y=at(1)), BAD), (dict(y=at(2)), BAD), (dict(out=at(8)), BAD), (dict(out=at(2, 16)), BAD), (dict(out=at(1)), BAD),
    (dict(out=at(5)), BAD), (dict(T=0, x=None, y=None), OK),
])
def test_residual_norm_refuses(bad, status):
    assert residual(**bad) == status


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("change,error,match", [
    (dict(x=t(9, 8, dtype=torch.float16)), TypeError, "bfloat16 or float32"),
    (dict(weight=t(8, 4, dtype=BF16)), TypeError, "weight: expected torch.float32"),
    (dict(weight=t(7, 4)), ValueError, "weight: expected shape"), (dict(bias=t(9)), ValueError, "bias: expected shape"),
    (dict(x=t(9, 16)[:, ::2]), ValueError, "rows must be contiguous"),
    (dict(x=t(1, 8).expand(9, 8)), ValueError, "rows overlap"),
    (dict(initial_state=t(1, 4, 8)), ValueError, "initial_state: expected shape"),
    (dict(cu_seqlens=[0, 9]), ValueError, "device int32 tensor"),
    (dict(cu_seqlens=torch.zeros(2, dtype=torch.int64)), TypeError, "cu_seqlens: expected torch.int32"),
    (dict(y=t(9, 9)), ValueError, "y: expected shape"), (dict(), ValueError, "device tensors"),
])
def test_conv_binding_checks(change, error, match):
    with pytest.raises(error, match=match):
        kda.conv_prefill(**{**dict(x=t(9, 8), weight=t(8, 4)), **change})


@pytest.mark.parametrize("change,error,match", [
    (dict(b=t(9, 2, 16, dtype=BF16)), TypeError, "b, c: expected"), (dict(b=t(9, 32)), ValueError, "b: expected shape"),
    (dict(c=t(9, 1, 16)), ValueError, "c: expected shape"), (dict(dt=t(9, 3)), ValueError, "dt: expected shape"),
    (dict(dt=t(9, 4, dtype=BF16)), TypeError, "dt: expected"), (dict(a=t(4, 1)), ValueError, "a: expected shape"),
    (dict(x=t(9, 4, 64)[..., :32]), ValueError, "rows must be contiguous"), (dict(skip=t(5)), ValueError, "skip"),
    (dict(initial_state=t(1, 4, 32, 16)), ValueError, "initial_state: expected shape"),
    (dict(workspace=t(512)), TypeError, "workspace"), (dict(), ValueError, "device tensors"),
])
def test_ssm_binding_checks(change, error, match):
    with pytest.raises(error, match=match):
        kda.ssm_prefill(**{**dict(x=t(9, 4, 32), dt=t(9, 4), a=t(4), b=t(9, 2, 16), c=t(9, 2, 16)), **change})


def test_step_and_norm_bindings_check():
    with pytest.raises(ValueError, match="state: expected shape"):
        kda.conv_step(t(3, 8), t(8, 4), t(3, 4, 8))
    with pytest.raises(ValueError, match="state is required"):
        kda.conv_step(t(3, 8), t(8, 4), None)
    with pytest.raises(ValueError, match="state: expected shape"):
        kda.ssm_step(t(3, 4, 32), t(3, 4), t(4), t(3, 2, 16), t(3, 2, 16), t(3, 4, 32, 16))
    with pytest.raises(ValueError, match="weight: expected shape"):
        kda.gated_norm(t(3, 4, 16), None, t(3, 16))
    with pytest.raises(ValueError, match="gate: expected shape"):
        kda.gated_norm(t(3, 4, 16), t(3, 4, 8), t(16))
    with pytest.raises(TypeError, match="residual: expected"):
        kda.residual_norm(t(3, 16), t(3, 16, dtype=BF16), t(16))
    with pytest.raises(ValueError, match="int32"):
        kda.conv_prefill(torch.empty(1, device="meta").expand(2 ** 31, 8), t(8, 4))
    with pytest.raises(ValueError, match="int32"):
        kda.conv_prefill(t(9, 1), torch.empty(1, device="meta").expand(1, 2 ** 32 + 4))
    with pytest.raises(ValueError, match="int32"):
        wide = torch.empty(1, device="meta").expand(9, 1, 2 ** 32 + 16)
        kda.ssm_prefill(t(9, 4, 32), t(9, 4), t(4), wide, wide)
    with pytest.raises(ValueError, match="int32"):
        kda.ssm_workspace(1, 9, 4, 2 ** 32 + 16, 32, "cpu")


def test_oracle_forms_agree():
    """The recurrence against its closed sum, the convolution against numpy's."""
    rng = np.random.default_rng(0)
    T, H, P, N = 11, 2, 3, 5
    x, b, c = rng.normal(size=(T, H, P)), rng.normal(size=(T, 1, N)), rng.normal(size=(T, 1, N))
    d, a = rng.uniform(0.1, 1, (T, H)), -rng.uniform(0.1, 2, H)
    y, _, states, _ = layer.ssm(x, d, a, b, c, cu=[0, 4, 11])
    for lo, hi in ((0, 4), (4, 11)):
        for t_ in range(lo, hi):
            for h in range(H):
                ref = sum(np.exp(a[h] * d[s + 1:t_ + 1, h].sum()) * d[s, h] * (c[t_, 0] @ b[s, 0]) * x[s, h]
                          for s in range(lo, t_ + 1))
                np.testing.assert_allclose(y[t_, h], ref, rtol=1e-12, atol=1e-13)
    w = rng.normal(size=(6, 4))
    z = rng.normal(size=(T, 6))
    out, _, end = layer.conv(z, w, None, [0, T], act=layer.NONE)
    for ch in range(6):
        np.testing.assert_allclose(out[:, ch], np.convolve(z[:, ch], w[ch, ::-1])[:T], atol=1e-12)
    np.testing.assert_array_equal(end[0], z[-3:])


def test_refusals_under_the_host_sanitizers():
    from gated_delta_rule_109_amd import build
    if not os.path.exists(build.HIPCC) or os.environ.get("KDA_LIB"):
        pytest.skip("needs hipcc, and is not run inside itself")
    lib = build.build_host_sanitized()
    env = dict(os.environ, LD_PRELOAD=build.san_runtime(), KDA_LIB=lib,
               ASAN_OPTIONS="detect_leaks=0:alloc_dealloc_mismatch=0:abort_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "refuse or workspace",
                        "tests/test_layer_abi.py"], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
