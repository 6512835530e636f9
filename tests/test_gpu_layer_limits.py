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


# ---- long walks ----------------------------------------------------------------------------

def cut(rng, T, n, outside):
    """Offsets of n sequences, cut anywhere, some of them empty; rows in front and behind."""
    inner = np.sort(rng.integers(outside[0], T - outside[1] + 1, n - 1))
    inner[n // 2] = inner[n // 2 - 1]
    return np.concatenate([[outside[0]], inner, [T - outside[1]]])


def conv_rows(x, w, b, cu, state, act):
    """layer.conv for long calls: the rows that each output needs, a shift at a time, in fp64 on
    the device; the same bounds. (Rows of no sequence: anything.)"""
    T, C = x.shape
    K = w.shape[1]
    t = torch.arange(T, device=DEV)
    seq = (torch.searchsorted(device_cu(cu), t.int(), right=True) - 1).clamp(0, len(cu) - 2)
    start = torch.tensor(cu, device=DEV)[seq]
    s = torch.zeros(T, C, dtype=torch.float64, device=DEV) + (b.double() if b is not None else 0.0)
    size = s.abs()
    for j in range(K):
        at = t - (K - 1) + j
        rows = x[at.clamp(min=0)].double()
        early = ((at < start) & (t >= start)).nonzero()[:, 0]
        rows[early] = state[seq[early], (at - start)[early] + K - 1].double() if state is not None else 0.0
        s += w[:, j].double() * rows
        size += (w[:, j].double() * rows).abs()
    bound = (K + 1) * layer.U * size
    if act:
        y = s * torch.sigmoid(s)
        return y, 1.1 * bound + y.abs() * (2 * s.abs() + 12) * layer.U
    return s, bound


@pytest.mark.parametrize("T,C,K,dtype,n", [
    (140001, 64, 4, BF16, 40), (800003, 12, 3, F32, 9), (36003, 1027, 4, BF16, 30), (16501, 4096, 4, BF16, 12),
    (43301, 777, 2, F32, 300), (9001, 7800, 4, F32, 1), (70001, 129, 3, BF16, 70)])
def test_conv_of_many_rows(T, C, K, dtype, n):
    """Calls large enough that a thread walks along 8 to 64 tokens: ragged ends, sequences that
    begin inside a walk, rows of every kind, states in place."""
    rng = np.random.default_rng(C)
    gen = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn(T, C, generator=gen, device=DEV).to(dtype)
    w, b = torch.randn(C, K, generator=gen, device=DEV) / 2, torch.randn(C, generator=gen, device=DEV)
    cu = cut(rng, T, n, (2, 3)) if n > 1 else np.array([2, T - 3])
    s = torch.randn(n, K - 1, C, generator=gen, device=DEV).to(dtype)
    state, y = s.clone(), torch.full((T, C), 7.0, dtype=dtype, device=DEV)
    kda.conv_prefill(x, w, b, cu_seqlens=device_cu(cu), initial_state=state, final_state=state, y=y)
    ref, bound = conv_rows(x, w, b, cu, s, True)
    inside = slice(int(cu[0]), int(cu[-1]))
    step = 2.0 ** -8 if dtype is BF16 else 2.0 ** -24
    err, tol = (y.double() - ref).abs(), bound * (1 + step) + step * ref.abs() + 1e-37
    assert (err[inside] <= tol[inside]).all()
    assert (y[:cu[0]] == 7).all() and (y[cu[-1]:] == 7).all()
    for i in range(n):
        rows = torch.cat([s[i], x[cu[i]:cu[i + 1]]])[-(K - 1):]
        assert torch.equal(state[i], rows)


@pytest.mark.parametrize("T,C,dtype,post,gate,scale", [
    (40001, 128, BF16, True, True, True), (70003, 20, F32, True, False, True), (10007, 512, BF16, False, True, False),
    (1301, 4096, BF16, True, True, True), (1027, 4099, BF16, True, True, True), (515, 8192, BF16, True, False, False),
    (1500, 2500, F32, True, True, True), (701, 16384, BF16, True, True, True), (600, 16383, BF16, False, True, True),
    (590, 16384, F32, True, True, True), (300, 5001, F32, True, False, True), (530, 16381, F32, True, True, False)])
def test_residual_norm_of_many_rows(T, C, dtype, post, gate, scale):
    """Calls in which a workgroup takes several rows, one after the other: in place and apart;
    rows of NaN, of infinities and of zeros change no row but their own."""
    gen = torch.Generator(device=DEV).manual_seed(C)
    x, r, g = (torch.randn(T, C, generator=gen, device=DEV).to(dtype) for _ in range(3))
    w, p, sc = (torch.randn(C, generator=gen, device=DEV) for _ in range(3))
    g, p, sc = (v if on else None for v, on in ((g, gate), (p, post), (sc, scale)))
    call = lambda x, r, **kw: kda.residual_norm(x, r, w, p, g, 2, sc, 0.5, 1e-5, **kw)  # noqa: E731
    out, y = call(x, r)
    ref, rb, yref, yb = layer.residual_norm(host(x), host(r), host(w), host(p), host(g), 2, host(sc), 0.5, float(np.float32(1e-5)))
    check(out, ref, rb, "residual")
    check(y, yref, yb, "y")
    same = r.clone()
    _, y2 = call(x, same, residual_out=same)
    assert torch.equal(same, out) and torch.equal(y2, y)
    x, r = x.clone(), r.clone()
    odd = [0, T // 3, T // 2, T - 2]
    x[odd[0]], x[odd[1]], r[odd[2]] = float("nan"), float("inf"), float("nan")
    x[odd[3]], r[odd[3]] = 0, 0
    out2, y2 = call(x, r)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[odd] = False
    assert torch.equal(out2[keep], out[keep]) and torch.equal(y2[keep], y[keep])
    assert torch.isnan(y2[odd[:3]]).any(1).all()
    assert (out2[odd[3]] == 0).all() and (y2[odd[3]] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gated_norm_rows_stay_apart(dtype):
    """As the residual norm's, in one workgroup and in others."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    for T, H, D in ((200, 3, 20), (40, 2, 512), (9, 3, 5000)):
        x, g = (torch.randn(T, H, D, generator=gen, device=DEV).to(dtype) for _ in range(2))
        w = torch.ones(D, device=DEV)
        for first in (False, True):
            y = kda.gated_norm(x, g, w, gate_first=first)
            x2 = x.clone()
            x2[T // 2, 1], x2[T // 2 + 1, 0], x2[T // 2 + 2, H - 1] = float("nan"), float("inf"), 0.0
            y2 = kda.gated_norm(x2, g, w, gate_first=first)
            keep = torch.ones(T, H, dtype=torch.bool, device=DEV)
            keep[T // 2, 1] = keep[T // 2 + 1, 0] = keep[T // 2 + 2, H - 1] = False
            assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[T // 2, 1]).all()
            assert torch.isnan(y2[T // 2 + 1, 0]).any() and (y2[T // 2 + 2, H - 1] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,H", [([700], 300), ([30, 620, 0, 330], 300), ([1500], 200), ([2, 1100, 500], 200)])
def test_ssm_of_long_walks(lengths, H, dtype):
    """Heads that fill the GPU: sequences of many chunks whole, or in segments of more than the 256
    tokens whose decays are made at a time."""
    s, s0, cu = layer_tests.ssm_inputs(lengths, (1, 2), H, 2, 16, 16, dtype, seed=H, rate=0.2)
    state = s0.clone()
    y, _ = kda.ssm_prefill(**s, cu_seqlens=device_cu(cu), initial_state=state, final_state=state)
    ref, bound, states, sbound = reference(s, cu, s0)
    check(y[cu[0]:cu[-1]], ref[cu[0]:cu[-1]], bound[cu[0]:cu[-1]], "y")
    check(state, states, sbound, "state")


def test_steps_and_residual_norm_past_32_bits():
    """Rows and states whose elements lie behind 2^31: as the last rows alone."""
    C, N = 1 << 20, 2100
    gen = torch.Generator(device=DEV).manual_seed(2)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    w = rand(C, 4)
    x, state = torch.zeros(N, C, dtype=BF16, device=DEV), torch.zeros(N, 3, C, dtype=BF16, device=DEV)
    x[-2:], state[-2:] = rand(2, C).to(BF16), rand(2, 3, C).to(BF16)
    small = state[-2:].clone()
    y = kda.conv_step(x, w, state)
    assert torch.equal(y[-2:], kda.conv_step(x[-2:].clone(), w, small)) and torch.equal(state[-2:], small)
    assert not y[:-2].any() and not state[1000].any()
    del state, y
    C, T = 16384, (1 << 31) // 16384 + 70
    rows = x.view(-1)[:T * C].view(T, C)
    rows.zero_()
    rows[-3:] = rand(3, C).to(BF16)
    w = rand(C)
    out, y = kda.residual_norm(rows, rows, w, post_weight=w, gate=rows, scale=w)
    tail = rows[-3:].clone()
    out2, y2 = kda.residual_norm(tail, tail, w, post_weight=w, gate=tail, scale=w)
    assert torch.equal(out[-3:], out2) and torch.equal(y[-3:], y2) and not y[-70:-3].any()
    del out, y, x, rows
    S, H, N, P = 1050, 32, 256, 256
    state = torch.zeros(S, H, N, P, device=DEV)
    state[-1] = rand(H, N, P)
    small = state[-1:].clone()
    x, b, c = rand(S, H, P).to(BF16), rand(S, 1, N).to(BF16), rand(S, 1, N).to(BF16)
    dt, a = torch.rand(S, H, generator=gen, device=DEV), -torch.ones(H, device=DEV)
    y = kda.ssm_step(x, dt, a, b, c, state)
    assert torch.equal(y[-1:], kda.ssm_step(x[-1:].clone(), dt[-1:].clone(), a, b[-1:].clone(), c[-1:].clone(), small)) \
        and torch.equal(state[-1:], small)
