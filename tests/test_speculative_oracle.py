"""Pins of the speculative-step oracle: trees against the chain recurrence of
the C oracle along every path, the verification's distribution in closed form,
the cache's rounding against definitions that do not share its code."""
import numpy as np
import pytest
import torch

from gated_delta_rule_109_amd.workloads import make_inputs
from oracle import reference, speculative


def tree_inputs(N, T, H, D, seed):
    inp = make_inputs(N * T, H, D, seed=seed, lengths=[T] * N, initial_state=True)
    return [x.reshape(N, T, *x.shape[1:]) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta)] + [inp.initial_state]


def random_parents(N, T, seed):
    rng = np.random.default_rng(seed)
    return np.array([[-1] + [int(rng.integers(0, i)) for i in range(1, T)] for _ in range(N)], np.int32)


def test_every_path_is_a_chain_of_the_recurrence_oracle():
    N, T, H, D = 2, 9, 2, 16
    q, k, v, g, beta, s0 = tree_inputs(N, T, H, D, 11)
    par = random_parents(N, T, 5)
    floor = float(np.float32(np.log(0.5)))         # the floor as a float argument carries it
    o = speculative.decode_tree(q, k, v, g, beta, s0, par, g_min=floor)
    for n in range(N):
        for i in range(T):
            path = [i]
            while par[n][path[0]] >= 0:
                path.insert(0, int(par[n][path[0]]))
            ref, fin, _ = reference.prefill(q[n, path], k[n, path], v[n, path], g[n, path], beta[n, path],
                                            initial_state=s0[n:n + 1], g_min=floor)
            np.testing.assert_allclose(o[n, i], ref[-1], rtol=1e-9, atol=1e-12)
            S, _, _ = speculative.commit_path(k, v, g, beta, s0, [path] * N, [len(path)] * N, g_min=floor)
            np.testing.assert_allclose(S[n], fin[0], rtol=1e-9, atol=1e-12)


def test_verification_returns_the_targets_distribution():
    """A root with two children drawn from q: over a grid of uniforms and every
    pair of draws, weighted by its probability, the first token has the
    target's distribution (lossless), up to the grid's 1 / 64."""
    p, q = np.array([0.5, 0.2, 0.3]), np.array([0.1, 0.6, 0.3])
    M = 64
    grid = (np.arange(M) + 0.5) / M
    got = np.zeros(3)
    for x1 in range(3):
        for x2 in range(3):
            # tests at the grid; the draw integrates exactly over its thresholds
            a1 = np.mean(grid * q[x1] < p[x1])
            r1 = np.maximum(p - q, 0)
            a2 = np.mean(grid * q[x2] * r1.sum() < r1[x2])
            r2 = np.maximum(p - (1 + r1.sum()) * q, 0)
            for u1 in (grid[grid * q[x1] < p[x1]][:1].tolist() + grid[~(grid * q[x1] < p[x1])][:1].tolist()):
                t1 = u1 * q[x1] < p[x1]
                for u2 in (grid[grid * q[x2] * r1.sum() < r1[x2]][:1].tolist()
                           + grid[~(grid * q[x2] * r1.sum() < r1[x2])][:1].tolist()):
                    t2 = u2 * q[x2] * r1.sum() < r1[x2]
                    w = q[x1] * q[x2] * (a1 if t1 else 1 - a1) * (a2 if t2 else 1 - a2)
                    for u0 in grid:
                        acc, path, tok = speculative.verify(
                            np.stack([p] * 3)[None], np.stack([q] * 3)[None], np.array([[0, x1, x2]]),
                            np.array([[u0, u1, u2]]), parents=np.array([[-1, 0, 0]]))
                        assert acc[0] == (2 if t1 or t2 else 1)
                        first = x1 if t1 else x2 if t2 else tok[0]
                        got[first] += w / M
                    if not t1 and not t2:
                        cum = np.cumsum(r2 / r2.sum())
                        assert tok[0] == np.searchsorted(cum, u0, side="right")
    assert np.abs(got - p).max() < 2 / M


@pytest.mark.parametrize("drafts", [(1, 2), (2, 0), (1, 1), (3, 2), (0, 0)])
def test_drafts_that_were_not_sampled_leave_the_targets_distribution(drafts):
    """A root with two children whose tokens were chosen without sampling (one
    may repeat or have no probability): over all uniforms the first token has
    the target's distribution. The tests' uniforms are integrated exactly over
    their thresholds, the draw's over a grid of 1 / 64."""
    p = np.array([0.5, 0.2, 0.3, 0.0])
    x1, x2 = drafts
    M = 64
    got = np.zeros(4)
    t1 = p[x1]                                               # accepted below these
    left = 1.0 - p[x1]
    r2 = p.copy(); r2[x1] = 0.0
    t2 = min(1.0, r2[x2] / left)
    for w1, u1 in ((t1, t1 / 2), (1 - t1, (1 + t1) / 2)):
        for w2, u2 in ((t2, t2 / 2), (1 - t2, (1 + t2) / 2)):
            if w1 * w2 == 0:
                continue
            for u0 in (np.arange(M) + 0.5) / M:
                acc, path, tok = speculative.verify(np.stack([p] * 3)[None], None, np.array([[0, x1, x2]]),
                                                    np.array([[u0, u1, u2]]), parents=np.array([[-1, 0, 0]]))
                first = (x1, x2)[path[0, 1] - 1] if acc[0] == 2 else tok[0]
                got[first] += w1 * w2 / M
    assert np.abs(got - p).max() < 2 / M


def test_rows_are_used_as_if_they_summed_to_one():
    """The header's example: given that the first token is rejected, the second
    is accepted below u = 0.5 of exact rows and below 0.32 of their bf16 values."""
    p = torch.tensor([0.9975, 0.00125, 0.00125])
    for row, below in ((p.double(), 0.5), (p.bfloat16().double(), 0.32)):
        row = row.numpy()
        for u2, accepted in ((below - 0.01, 2), (below + 0.01, 1)):
            acc, _, _ = speculative.verify(np.stack([row] * 3)[None], None, np.array([[0, 0, 1]]),
                                           np.array([[0.5, 0.999, u2]]), parents=np.array([[-1, 0, 0]]))
            assert acc[0] == accepted


def test_verification_by_hand():
    p = np.array([[[0.25, 0.5, 0.25, 0.0], [0.0, 0.0, 1.0, 0.0], [0.125, 0.125, 0.25, 0.5]]])
    tok = np.array([[9, 1, 2]])
    # chain without draft rows: 0.4 < p(1) = 0.5, then 0.9 < p(2) = 1; the last row's draw
    acc, path, nxt = speculative.verify(p, None, tok, np.array([[0.5, 0.4, 0.9]]))
    assert (acc[0], path[0].tolist(), nxt[0]) == (3, [0, 1, 2], 3)
    # rejected at once: 0.5 < 0.5 is false; the draw is from row 0 without token 1
    acc, path, nxt = speculative.verify(p, None, tok, np.array([[0.5, 0.5, 0.9]]))
    assert (acc[0], path[0].tolist(), nxt[0]) == (1, [0, -1, -1], 2)
    acc, _, nxt = speculative.verify(p, None, tok, np.array([[0.5, 0.5, 0.9]]), num_nodes=[0])
    assert (acc[0], nxt[0]) == (0, -1)


def test_e4m3_table_and_int8_steps():
    t = speculative.e4m3_values()
    assert t[0x7e] == 448 and np.isnan(t[0x7f]) and t[1] == 2.0 ** -9 and t[0x38] == 1.0 and t[0xb8] == -1.0
    x = np.zeros((1, 1, 16, 16), np.float32)
    x[0, 0, 0, :4] = [127.0, 0.5, 1.5, -2.5]
    y, c = speculative.quantise(x, False)
    assert y[0, 0, :4].tolist() == [127, 0, 2, -2] and c[0, 0, 0] == 127 and c[0, 0, 1] == 0
    x[0, 0, 0, 0] = np.nextafter(np.float32(127), np.float32(200))
    assert speculative.quantise(x, False)[1][0, 0, 0] == 128
    y, c = speculative.quantise(x, True)
    assert c[0, 0, 0] == 126 and y[0, 0, 0] == 256.0


@pytest.mark.parametrize("e4m3", [False, True])
def test_quantisation_is_the_nearest_value(e4m3):
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((3, 2, 16, 16)) * 10.0 ** rng.integers(-6, 6, (3, 2, 16, 1))).astype(np.float32)
    y, c = speculative.quantise(x, e4m3)
    values = speculative.e4m3_values() if e4m3 else np.arange(-127.0, 128.0)
    values = values[np.isfinite(values)]
    b = x.reshape(3, 2, -1, 32).astype(np.float64) / 2.0 ** (c.astype(np.float64) - 127)[..., None]
    assert np.abs(b).max() <= values.max()
    near = np.abs(b[..., None] - values).min(-1)
    assert (np.abs(b - y.reshape(b.shape)) == near).all()
