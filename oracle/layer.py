"""fp64 references of the operators around a recurrence (short convolution,
state-space scan, norms with gate and residual): TEST INFRASTRUCTURE ONLY (see
oracle/__init__.py).

Plain numpy, one formula per step, token by token; with each result the bound
on the error of arithmetic in u = 2^-24 (fp32) that the tests count, element by
element, without the rounding of the result to its storage type.
"""
import numpy as np

U = 2.0 ** -24
NONE, SILU, SIGMOID = 0, 1, 2


def activate(x, act):
    if act == NONE:
        return np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        s = 1.0 / (1.0 + np.exp(-np.asarray(x, np.float64)))
    return x * s if act == SILU else s


def activate_bound(x, act, err):
    """Error of act(x) given x within err: act' is at most 1.1; the exponential
    of an argument rounded to fp32 is within (|x| + 4) u of its value and the
    sum, the reciprocal and the product round once or twice each."""
    if act == NONE:
        return err
    return 1.1 * err + np.abs(activate(x, act)) * (2 * np.abs(x) + 12) * U


def offsets(lengths, first=0):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64) + first


def conv(x, weight, bias, cu, initial=None, act=SILU):
    """(y, bound, states): y [T,C] (0 outside the sequences), states [n,K-1,C]."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    T, C = x.shape
    K = w.shape[1]
    b = np.zeros(C) if bias is None else np.asarray(bias, np.float64)
    y, bound = np.zeros((T, C)), np.zeros((T, C))
    states = np.zeros((len(cu) - 1, K - 1, C))
    for n in range(len(cu) - 1):
        past = np.zeros((K - 1, C)) if initial is None else np.asarray(initial[n], np.float64)
        rows = np.concatenate([past, x[cu[n]:cu[n + 1]]])
        L = cu[n + 1] - cu[n]
        for t in range(L):
            s = b + (w.T * rows[t:t + K]).sum(0)
            size = np.abs(b) + (np.abs(w.T) * np.abs(rows[t:t + K])).sum(0)
            y[cu[n] + t] = activate(s, act)
            bound[cu[n] + t] = activate_bound(s, act, (K + 1) * U * size)
        states[n] = rows[L:]
    return y, bound, states


def softplus(v):
    return np.logaddexp(0.0, np.asarray(v, np.float64))


def ssm(x, dt, a, b, c, skip=None, dt_bias=None, soft=False, cu=None, initial=None, product=0.0):
    """(y, y bound, states, state bound): x [T,H,P], b, c [T,G,N]. `product` is
    the relative error of one product of an output besides fp32 rounding.

    Bounds, with M the state of the absolute values: a step's size d is within
    e_d = (|v| + 8) u of its value (v = dt + dt_bias rounds, then a logarithm of
    an exponential), its decay f = exp(d a) within e_f = |d a| (e_d + 3 u) + 4 u,
    and S <- f S + d b x^T rounds three times more:
        E <- f E + f M (e_f + 2 u) + |d b x| (e_d + 4 u).
    (In chunks each pair of tokens takes its decay at once, from sums in fp64:
    no more.) A sum of N products is within (N + 4) u of its terms' sizes."""
    x, b, c = (np.asarray(z, np.float64) for z in (x, b, c))
    T, H, P = x.shape
    G, N = b.shape[1:]
    v = np.asarray(dt, np.float64) + (0.0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    d = softplus(v) if soft else v
    ed = (np.abs(v) + 8) * U
    da = d * np.asarray(a, np.float64)
    f = np.exp(da)
    ef = np.abs(da) * (ed + 3 * U) + 4 * U
    cu = [0, T] if cu is None else cu
    y, yb = np.zeros((T, H, P)), np.zeros((T, H, P))
    states, sb = np.zeros((len(cu) - 1, H, N, P)), np.zeros((len(cu) - 1, H, N, P))
    per = H // G
    D = np.zeros(H) if skip is None else np.asarray(skip, np.float64)
    for n in range(len(cu) - 1):
        S = np.zeros((H, N, P)) if initial is None else np.asarray(initial[n], np.float64).copy()
        M, E = np.abs(S), np.zeros((H, N, P))
        for t in range(cu[n], cu[n + 1]):
            bt, ct = b[t].repeat(per, 0), c[t].repeat(per, 0)
            ft, fe = f[t][:, None, None], ef[t][:, None, None]
            w = (d[t][:, None] * bt)[..., None] * x[t][:, None, :]
            E = ft * E + ft * M * (fe + 2 * U) + np.abs(w) * (ed[t][:, None, None] + 4 * U)
            S, M = ft * S + w, ft * M + np.abs(w)
            sk = D[:, None] * x[t]
            y[t] = (S * ct[..., None]).sum(1) + sk
            size = (M * np.abs(ct)[..., None]).sum(1)
            yb[t] = (E * np.abs(ct)[..., None]).sum(1) + size * ((N + 4) * U + product) + 2 * U * np.abs(sk)
        states[n], sb[n] = S, E
    return y, yb, states, sb


def _norm(v, bound, eps):
    """norm(v) and its bound, v within `bound`: the mean of squares is within
    (D + 2) u of its value and twice the relative error of v, its root half of it."""
    D = v.shape[-1]
    ms = (v * v).mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(ms + eps)
    dms = 2 * (np.abs(v) * bound).mean(-1, keepdims=True) + (bound * bound).mean(-1, keepdims=True) + (D + 2) * U * ms
    rel = 0.5 * dms / (ms + eps) + 4 * U
    return v * r, (bound + np.abs(v) * (1.1 * rel + U)) * r


def gated_norm(x, gate, weight, act=SIGMOID, gate_first=False, eps=1e-6):
    """(y, bound) over [T,H,D]."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    g = np.ones_like(x) if gate is None else activate(np.asarray(gate, np.float64), act)
    gb = np.zeros_like(x) if gate is None else activate_bound(np.asarray(gate, np.float64), act, 0.0)
    if gate_first:
        v = x * g
        y, b = _norm(v, np.abs(x) * gb + U * np.abs(v), eps)
        return y * w, b * np.abs(w) + U * np.abs(y * w)
    y, b = _norm(x, np.zeros_like(x), eps)
    return y * w * g, b * np.abs(w * g) + np.abs(y * w) * gb + 2 * U * np.abs(y * w * g)


def residual_norm(x, residual, weight, post=None, gate=None, act=SIGMOID, scale=None, alpha=1.0, eps=1e-6):
    """(residual', bound, y, bound) over [T,C]."""
    v = np.asarray(x, np.float64)
    b = np.zeros_like(v)
    if post is not None:
        v, b = _norm(v, b, eps)
        p = np.asarray(post, np.float64)
        v, b = v * p, b * np.abs(p) + U * np.abs(v * p)
    if gate is not None:
        z = np.asarray(gate, np.float64)
        g, gb = activate(z, act), activate_bound(z, act, 0.0)
        v, b = v * g, b * np.abs(g) + np.abs(v) * gb + U * np.abs(v * g)
    k = alpha * (1.0 if scale is None else np.asarray(scale, np.float64))
    r = 0.0 if residual is None else np.asarray(residual, np.float64)
    out = r + k * v
    b = np.abs(k) * b + 2 * U * np.abs(k * v) + U * np.abs(out)
    y, yb = _norm(out, b, eps)
    w = np.asarray(weight, np.float64)
    return out, b, y * w, yb * np.abs(w) + U * np.abs(y * w)
