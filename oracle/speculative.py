"""fp64 reference of one speculative step over the recurrent state, and of the
8-bit state cache: TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

Trees and paths run the token recurrence along each node's path, one outer
product after the other (nothing of the kernels' unrolled form, except in the
error bounds). The verification walks one sequence's tree at a time with the
residual row written out. The cache rounds exact quotients.
"""
import numpy as np

U32 = 2.0 ** -24          # half a step of fp32, relative


def parents_of(parents, T):
    """Row of parents as used: chains for None, -1 for values outside [-1, i - 1]."""
    if parents is None:
        return np.arange(T) - 1
    p = np.asarray(parents).copy()
    i = np.arange(T)
    p[(p < 0) | (p >= i)] = -1
    return p


def alpha_of(g, g_min, H, D, N, T):
    """Decay [N, T, H, D] from the log-decay in any gate layout (None: 1)."""
    if g is None:
        return np.ones((N, T, H, D))
    a = np.exp(np.clip(np.asarray(g, np.float64), np.float64(np.float32(g_min)), 0.0))
    return np.broadcast_to(a if a.ndim == 4 else a[..., None], (N, T, H, D))


def step(S, k, v, a, b):
    """One token on S [.., D, D]: decay, retrieve, write."""
    S = S * a[..., None]
    d = b[..., None] * (v - np.einsum("...cd,...c->...d", S, k))
    return S + k[..., None] * d[..., None, :], d


def decode_tree(q, k, v, g, beta, state, parents=None, num_nodes=None, scale=1.0, g_min=np.log(0.5)):
    """o [N, T, H, D] fp64 (NaN rows where a sequence has no such node)."""
    q, k, v, beta, state = (np.asarray(x, np.float64) for x in (q, k, v, beta, state))
    N, T, H, D = q.shape
    a = alpha_of(g, g_min, H, D, N, T)
    o = np.full((N, T, H, D), np.nan)
    for n in range(N):
        par = parents_of(None if parents is None else parents[n], T)
        nt = T if num_nodes is None else int(np.clip(num_nodes[n], 0, T))
        states = []
        for i in range(nt):
            S = state[n] if par[i] < 0 else states[par[i]]
            S, _ = step(S, k[n, i], v[n, i], a[n, i], beta[n, i])
            states.append(S)
            o[n, i] = scale * np.einsum("hcd,hc->hd", S, q[n, i])
    return o


def commit_path(k, v, g, beta, state, path, accept, g_min=np.log(0.5)):
    """(state after the path [N, H, D, D], largest |S column| 2-norm + |d| on the
    way [N, H, D], the path lengths)."""
    k, v, beta = (np.asarray(x, np.float64) for x in (k, v, beta))
    S = np.array(state, np.float64)
    N, T, H, D = k.shape
    a = alpha_of(g, g_min, H, D, N, T)
    size = np.sqrt((S * S).sum(-2))
    lengths = np.zeros(N, int)
    for n in range(N):
        for j in range(int(np.clip(accept[n], 0, T))):
            i = int(path[n][j])
            if not 0 <= i < T:
                break
            S[n], d = step(S[n], k[n, i], v[n, i], a[n, i], beta[n, i])
            size[n] = np.maximum(size[n], np.sqrt((S[n] ** 2).sum(-2)) + np.abs(d))
            lengths[n] = j + 1
    return S, size, lengths


def tree_bound(q, k, v, g, beta, state, par, nt, scale, g_min, product):
    """How far fp32 arithmetic may leave one sequence's outputs from exact ones
    ([nt, H, D]), where each product of the unrolled form (see the header) has
    the relative error `product` and sums keep fp32: with abs values of every
    term in place of the terms,
      bound_d = |L^-1| gamma (|b| + |beta A| |d|)        L = I + beta A
      bound_o = scale (gamma (|q E| |S| + |B| |d|) + |B| bound_d)
    gamma = product + (D + 6 T + 16) 2^-24: D + T terms a sum, a path of at most
    T decays of 5 roundings each. Doubled for what is quadratic in gamma."""
    q, k, v, beta, state = (np.asarray(x, np.float64) for x in (q, k, v, beta, state))
    T, H, D = k.shape
    a = alpha_of(None if g is None else np.asarray(g)[None], g_min, H, D, 1, T)[0]
    gamma = product + (D + 6 * T + 16) * U32
    out = np.zeros((nt, H, D))
    for h in range(H):
        E = np.ones((nt, D))
        ratio = {}
        for i in range(nt):
            r, j = a[i, h].copy(), par[i]
            while j >= 0:
                ratio[i, j] = r.copy()
                r = r * a[j, h]
                j = par[j]
            E[i] = r
        A, Aabs, B, Babs = (np.zeros((nt, nt)) for _ in range(4))
        for (i, j), r in ratio.items():
            A[i, j] = (k[i, h] * k[j, h] * r).sum()
            Aabs[i, j] = np.abs(k[i, h] * k[j, h] * r).sum()
            B[i, j] = (q[i, h] * k[j, h] * r).sum()
            Babs[i, j] = np.abs(q[i, h] * k[j, h] * r).sum()
        for i in range(nt):
            B[i, i], Babs[i, i] = (q[i, h] * k[i, h]).sum(), np.abs(q[i, h] * k[i, h]).sum()
        bt = beta[:nt, h, None]
        S, Sabs = state[h], np.abs(state[h])
        inv = np.linalg.inv(np.eye(nt) + bt * A)
        d = inv @ (bt * (v[:nt, h] - (k[:nt, h] * E) @ S))
        babs = np.abs(bt) * (np.abs(v[:nt, h]) + (np.abs(k[:nt, h]) * E) @ Sabs)
        bd = np.abs(inv) @ (gamma * (babs + (np.abs(bt) * Aabs) @ np.abs(d)))
        out[:, h] = 2 * abs(scale) * (gamma * ((np.abs(q[:nt, h]) * E) @ Sabs + Babs @ np.abs(d)) + np.abs(B) @ bd)
    return out


def weights(x):
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        return np.where((x > 0) & np.isfinite(x), x, 0.0)


def verify(target, draft, tokens, uniforms, parents=None, num_nodes=None):
    """(accept [N], path [N, T], next_token [N])."""
    N, T, V = target.shape
    accept, path, token = np.zeros(N, np.int32), np.full((N, T), -1, np.int32), np.full(N, -1, np.int32)
    u = np.asarray(uniforms, np.float64)
    for n in range(N):
        par = parents_of(None if parents is None else parents[n], T)
        nt = T if num_nodes is None else int(np.clip(num_nodes[n], 0, T))
        if nt == 0:
            continue
        walked = [0]
        while True:
            cur = walked[-1]
            p = weights(target[n, cur])
            q = None if draft is None else weights(draft[n, cur])
            r, c, took, spent = p.copy(), 1.0, None, 0.0
            for i in range(cur + 1, nt):
                if par[i] != cur:
                    continue
                x = int(tokens[n, i])
                known = 0 <= x < V
                rx = r[x] if known else 0.0
                qx = 1.0 if q is None else q[x] if known else 0.0
                if u[n, i] * qx * c < rx:
                    took = i
                    break
                if q is None:
                    c -= rx
                    if known:
                        r[x] = 0.0
                else:
                    spent += c
                    r = np.maximum(p - spent * q, 0.0)
                    c = r.sum()
            if took is None:
                break
            walked.append(took)
        if not r.sum() > 0:
            r = p
        cum = np.cumsum(r)
        if cum[-1] > 0:
            goal = max(u[n, 0], 0.0) * cum[-1]
            past = np.nonzero((cum > goal) & (r > 0))[0]
            token[n] = past[0] if len(past) else np.nonzero(r)[0][-1]
        accept[n] = len(walked)
        path[n, :len(walked)] = walked
    return accept, path, token


def e4m3_values():
    """The 256 values of the 8-bit float format (code 0x7f / 0xff: NaN)."""
    out = np.zeros(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = np.nan if b & 127 == 127 else m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = -x if b & 128 else x
    return out


def quantise(x, e4m3):
    """fp32 states [.., D, D] -> (values as fp64 multiples of the step [.., D*D],
    scale codes [.., D*D/32]), from exact quotients."""
    x = np.asarray(x, np.float32).astype(np.float64)
    b = x.reshape(*x.shape[:-2], -1, 32)
    top = 448.0 if e4m3 else 127.0
    amax = np.where(np.isfinite(b), np.abs(b), 0.0).max(-1)
    e = np.full(amax.shape, -127)
    for i in np.ndindex(amax.shape):
        while amax[i] > top * 2.0 ** e[i]:
            e[i] += 1
    y = np.clip(b * 2.0 ** -e[..., None].astype(np.float64), -top, top)
    if e4m3:
        table = e4m3_values()[:127]                       # 0 .. 448
        mag = np.abs(np.nan_to_num(y))
        hi = np.minimum(np.searchsorted(table, mag, side="left"), 126)
        lo = np.maximum(hi - 1, 0)
        up, down = table[hi] - mag, mag - table[lo]
        pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)   # even codes have even mantissas
        pick = np.where(table[hi] == mag, hi, pick)
        y = np.where(np.isnan(b), np.nan, np.sign(y) * table[pick])
    else:
        y = np.where(np.isnan(b), 0.0, np.rint(np.nan_to_num(y)))
    return y.reshape(*x.shape[:-2], -1), (e + 127).astype(np.uint8)


def dequantise(y, code):
    """What cached values stand for: y [.., D*D] times 2^(code - 127), fp64, no
    larger than the largest fp32 number."""
    b = np.asarray(y, np.float64).reshape(*code.shape, 32)
    top = float(np.finfo(np.float32).max)
    return np.clip(b * 2.0 ** (code.astype(np.float64) - 127)[..., None], -top, top).reshape(np.shape(y))
