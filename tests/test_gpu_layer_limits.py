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
