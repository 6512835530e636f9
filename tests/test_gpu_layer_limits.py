"""The operators around a recurrence on the GPU where their numbers reach limits: factors of
products that cancel, states that grow, and the long loops of calls of many rows. Against the
fp64 oracle, closed forms, or the same rows in other calls, to the bit."""
import numpy as np
import pytest
import torch

import test_gpu_layer as layer_tests
from gated_delta_rule_109_amd import kda
from oracle import layer

pytestmark = pytest.mark.gpu
DEV, BF16, F32 = layer_tests.DEV, layer_tests.BF16, layer_tests.F32
dev, host, check, device_cu = layer_tests.dev, layer_tests.host, layer_tests.check, layer_tests.device_cu


# ---- the scan's own numbers --------------------------------------------------------------

def exact_values(rng, shape, off):
    """Numbers of 24 bits in [1, 2), and others within `off` of them: multiples of 2^-23, so that
    sums of a few of them below 2 are exact in fp32 whatever their order."""
    k = rng.integers(1 << 23, (1 << 24) - off, shape)
    return k * 2.0 ** -23, (k + rng.integers(-off, off, shape)).clip(1 << 23, (1 << 24) - 1) * 2.0 ** -23


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,P,T", [(16, 16, 40), (32, 64, 150), (128, 128, 200), (256, 48, 70), (64, 32, 1100)])
def test_ssm_factors_keep_24_bits(dtype, N, P, T):
    """Outputs that are differences of nearly equal products: of two rows of the state in front,
    and of two tokens of the prompt. The decay is 1, b, c and x are 0, 1 or -1, so all products
    and sums are exact, and so is the output up to its rounding: equal to the bit."""
    rng = np.random.default_rng(N + T)
    H, off = 3, 1 << 10
    p, q = exact_values(rng, (H, P), off)
    d, e = exact_values(rng, H, off)
    s0 = np.zeros((1, H, N, P))
    s0[0, :, 2], s0[0, :, 11] = p, q
    x, b, c, dt = np.zeros((T, H, P)), np.zeros((T, 1, N)), np.zeros((T, 1, N)), np.zeros((T, H))
    b[:, 0, 5] = 1
    x[3], x[9] = 1, -1
    dt[3], dt[9] = d, e
    c[:, 0, 5] = 1                                   # tokens: d, then d - e
    c[1::2] = 0
    c[1::2, 0, 2], c[1::2, 0, 11] = 1, -1            # every other one: the state in front
    want = np.zeros((T, H, P))
    want[3:] = d[None, :, None]
    want[9:] = (d - e)[None, :, None]
    want[1::2] = p - q
    want[0] = 0
    y, end = kda.ssm_prefill(dev(x, dtype), dev(dt), torch.zeros(H, device=DEV), dev(b, dtype), dev(c, dtype),
                             initial_state=dev(s0))
    assert torch.equal(y, dev(want, dtype))
    s0[0, :, 5] = (d - e)[:, None]
    assert torch.equal(end, dev(s0))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [70, 900])
def test_ssm_largest_finite_factors(dtype, T):
    """A state and a step size near the largest finite number, which rounds to infinity in bf16:
    what b, c and x make small, and what they leave out, is finite. Products by powers of 2: exact."""
    N, P, big = 16, 16, float(np.finfo(np.float32).max)
    s0 = np.zeros((1, 2, N, P))
    s0[0, 0, 2], s0[0, 0, 3], s0[0, 1, 4] = big, -big, 1.5
    x, b, c, dt = np.zeros((T, 2, P)), np.zeros((T, 1, N)), np.zeros((T, 1, N)), np.zeros((T, 2))
    x[5], b[5, 0, 5], dt[5, 1] = 2.0 ** -10, 1, big
    c[:, 0, 5] = 1
    c[::2, 0, 5], c[::2, 0, 2], c[::2, 0, 4] = 0, 2.0 ** -10, 1
    want = np.zeros((T, 2, P))
    want[5:, 1] = big * 2.0 ** -10
    want[::2, 0], want[::2, 1] = big * 2.0 ** -10, 1.5
    y, end = kda.ssm_prefill(dev(x, dtype), dev(dt), torch.zeros(2, device=DEV), dev(b, dtype), dev(c, dtype),
                             initial_state=dev(s0))
    assert torch.equal(y, dev(want, dtype))
    s0[0, 1, 5] = big * 2.0 ** -10
    assert torch.equal(end, dev(s0))


# ---- states that grow ---------------------------------------------------------------------

def reference(s, cu, s0):
    """The oracle with the bounds of fp32 arithmetic alone."""
    return layer.ssm(host(s["x"]), host(s["dt"]), host(s["a"]), host(s["b"]), host(s["c"]), host(s["skip"]),
                     host(s["dt_bias"]), s["dt_softplus"], cu, host(s0))


def growing(kind, lengths, H, N, P, dtype, seed):
    """Inputs whose decay rates are positive (1): a sequence's step sizes are its logarithms."""
    s, s0, cu = layer_tests.ssm_inputs(lengths, (1, 2), H, 1, N, P, dtype, soft=False, seed=seed)
    s["a"] = torch.ones(H, device=DEV)
    for n, L in enumerate(lengths):
        x, dt, first = s["x"][cu[n]:cu[n + 1]], s["dt"][cu[n]:cu[n + 1]], s0[n]
        if kind == "zero until the end":          # e^2 a token; nothing to multiply but for the last 30
            dt.fill_(2.0)
            first.zero_()
            x[:max(L - 30, 0)] = 0
        elif kind == "small states":              # e^132 over the first tokens, then as it is
            dt.zero_()
            dt[:33] = 4.0
            first *= 1e-32
            x[:30] = 0
        else:                                     # up and down, by at most e^36 from any token to any other
            c = np.random.default_rng(seed + n).uniform(-18, 18, (L + 1, H))
            dt.copy_(dev(np.diff(c, axis=0)))
    return s, s0, cu


GROWING = [([200, 3, 64], 2, 32, 48), ([150, 131], 2, 128, 128), ([140], 1, 256, 80), ([170], 2, 16, 16),
           ([133], 1, 64, 144), ([900, 5, 450], 1, 16, 32), ([700], 1, 64, 16)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["zero until the end", "small states", "up and down"])
@pytest.mark.parametrize("lengths,H,N,P", GROWING)
def test_ssm_states_that_grow_far(lengths, H, N, P, kind, dtype):
    """Growth by more than e^88 within a chunk and within a segment: where the recurrence stays
    finite, so do outputs and states, in place and apart."""
    s, s0, cu = growing(kind, lengths, H, N, P, dtype, N + P)
    state = s0.clone()
    y, _ = kda.ssm_prefill(**s, cu_seqlens=device_cu(cu), initial_state=state, final_state=state)
    ref, bound, states, sbound = reference(s, cu, s0)
    check(y[cu[0]:cu[-1]], ref[cu[0]:cu[-1]], bound[cu[0]:cu[-1]], "y")
    check(state, states, sbound, "state")
    y2, end = kda.ssm_prefill(**s, cu_seqlens=device_cu(cu), initial_state=s0)
    assert torch.equal(y2[cu[0]:cu[-1]], y[cu[0]:cu[-1]]) and torch.equal(end, state)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["prompt", "steps"])
def test_ssm_single_tokens_that_grow_far(form, dtype):
    """Factors of e^100 and e^150, which are infinite in fp32, on states of 0 and small ones."""
    H, N, P, L = 2, 32, 48, 70
    s, s0, _ = layer_tests.ssm_inputs([L], (0, 0), H, 1, N, P, dtype, soft=False, seed=3)
    s["a"] = torch.ones(H, device=DEV)
    s["dt"].mul_(0.05)
    s["dt"][20], s["dt"][L - 1, 0] = 100.0, 150.0
    s0 *= 1e-34
    s0[:, :, ::2] = 0
    s0[:, 0] = 0
    s["x"][:L - 1] = 0
    ref, bound, states, sbound = reference(s, [0, L], s0)
    if form == "prompt":
        y, state = kda.ssm_prefill(**s, initial_state=s0)
    else:
        state = s0.clone()
        row = lambda t: {k: v[t:t + 1].clone() if k in ("x", "b", "c", "dt") else v for k, v in s.items()}  # noqa: E731
        y = torch.cat([kda.ssm_step(state=state, **row(t)) for t in range(L)])
    check(y, ref, bound, "y")
    check(state, states, sbound, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ssm_growth_keeps_what_is_not_finite_from_earlier_tokens(dtype):
    """As without growth: x spoils its column, b and dt their head, c its token."""
    T, H, P = 150, 4, 48
    s, s0, _ = layer_tests.ssm_inputs([T], (0, 0), H, 4, 32, P, dtype, soft=False, seed=8)
    s["a"] = torch.ones(H, device=DEV)
    s["dt"].fill_(0.5)
    s0 *= 1e-20
    s["x"] *= 1e-20
    y, end = kda.ssm_prefill(**s, initial_state=s0)
    s["x"][90, 0, 5], s["x"][91, 0, 20], s["x"][30, 0, 21] = float("nan"), float("inf"), float("-inf")
    s["b"][100, 1, 3] = float("nan")
    s["dt"][70, 2] = float("nan")
    s["c"][33, 3, 9] = float("nan")
    y2, end2 = kda.ssm_prefill(**s, initial_state=s0)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[90:, 0, 5] = bad[91:, 0, 20] = bad[30:, 0, 21] = True
    bad[100:, 1] = bad[70:, 2] = bad[33, 3] = True
    assert (~torch.isfinite(y2[bad])).all()
    assert torch.equal(y2[~bad], y[~bad])
    sbad = torch.zeros_like(end, dtype=torch.bool)
    sbad[:, 0, :, [5, 20, 21]] = sbad[:, 1, 3] = sbad[:, 2] = True
    assert (~torch.isfinite(end2[sbad])).all()
    assert torch.equal(end2[~sbad], end[~sbad])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 70, 900])
def test_ssm_rates_of_minus_infinity(dtype, T):
    """A rate of -infinity ends the state at every token, as the lowest finite rate does: the same
    bits, finite outputs and final states, whether or not the last chunk is whole."""
    s, s0, _ = layer_tests.ssm_inputs([T], (0, 0), 2, 1, 32, 48, dtype, soft=False, seed=T)
    s["dt"] += 0.01
    s["a"] = dev([-np.finfo(np.float32).max, -1.0])
    y, end = kda.ssm_prefill(**s, initial_state=s0)
    ref, bound, states, sbound = reference(s, [0, T], s0)
    check(y, ref, bound, "y")
    check(end, states, sbound, "state")
    s["a"][0] = -float("inf")
    y2, end2 = kda.ssm_prefill(**s, initial_state=s0)
    assert torch.equal(y2, y) and torch.equal(end2, end)
    if T == 1:
        state = s0.clone()
        check(kda.ssm_step(state=state, **s), ref, bound, "y of a step")
        check(state, states, sbound, "state of a step")
