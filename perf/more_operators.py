"""Cases, plain forms and exact values of the operators around a recurrence over packed sequences, and of the second
recurrence of that family: the short causal convolution before it, the selective state-space scan, the norm of the
heads' outputs with the output gate, and the norms before and after a block with its gate and residual scale.

``own = False`` computes the operators from elementary torch operations; ``own = True`` calls the library.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 64


# ---- cases ---------------------------------------------------------------------
# The keys: op; T tokens of N packed sequences (cut at random places) or N sequences of one token each (steps);
# C channels; K width of the convolution; H heads of P channels, states of S rows, G groups that share B and C;
# D values under one norm; cached: sequences start from states of an earlier call.

def _conv_case(name, T, N, C, K, dtype, act, bias, cached):
    return {"name": name, "op": "conv", "T": T, "N": N, "C": C, "K": K, "dtype": dtype, "act": act, "bias": bias,
            "cached": cached}


def _conv_step_case(name, N, C, K, dtype, act, bias):
    return {"name": name, "op": "conv_step", "N": N, "C": C, "K": K, "dtype": dtype, "act": act, "bias": bias}


def _ssm_case(name, T, N, H, P, S, G, dtype, cached, skip=True):
    return {"name": name, "op": "ssm", "T": T, "N": N, "H": H, "P": P, "S": S, "G": G, "dtype": dtype,
            "cached": cached, "skip": skip}


def _ssm_step_case(name, N, H, P, S, G, dtype, skip=True):
    return {"name": name, "op": "ssm_step", "N": N, "H": H, "P": P, "S": S, "G": G, "dtype": dtype, "skip": skip}


def _gated_case(name, T, H, D, dtype, act, first, shared):
    return {"name": name, "op": "gated", "T": T, "H": H, "D": D, "dtype": dtype, "act": act, "gate_first": first,
            "shared": shared}


def _residual_case(name, T, C, dtype, post, gate, scale):
    return {"name": name, "op": "residual", "T": T, "C": C, "dtype": dtype, "post": post, "gate": gate,
            "scale": scale}


def listed():
    return [
        # q, k and v of a prompt of 8192 tokens, 32 heads of 128, convolved together before the recurrence
        _conv_case("conv 8192x12288", 8192, 1, 12288, 4, "bf16", "silu", False, False),
        # appended parts of nine sequences, odd sizes, from cached rows
        _conv_case("conv 3001x777 f32", 3001, 9, 777, 3, "f32", "silu", True, True),
        # the decode batch of 256 sequences
        _conv_step_case("conv step 256x12288", 256, 12288, 4, "bf16", "silu", False),
        # one user's next token: latency
        _conv_step_case("conv step 1x777 f32", 1, 777, 3, "f32", "silu", True),
        # a prompt of 8192 tokens, 32 heads of 128
        _ssm_case("ssm 8192 32x128x128", 8192, 1, 32, 128, 128, 8, "bf16", False),
        # appended parts of nine sequences in fp32, odd sizes, from cached states
        _ssm_case("ssm 3001 6x48x32 f32", 3001, 9, 6, 48, 32, 1, "f32", True),
        # the decode batch
        _ssm_step_case("ssm step 256 32x128x128", 256, 32, 128, 128, 8, "bf16"),
        # one user's next token
        _ssm_step_case("ssm step 1 32x128x128", 1, 32, 128, 128, 8, "bf16"),
        # the heads' outputs of the prompt, normalised and gated
        _gated_case("gated norm 8192x32x128", 8192, 32, 128, "bf16", "sigmoid", False, True),
        # odd sizes in fp32, the gate before the norm
        _gated_case("gated norm 777x5x100 f32", 777, 5, 100, "f32", "silu", True, False),
        # between two blocks of the prompt: both norms, gate and scale
        _residual_case("residual norm 8192x4096", 8192, 4096, "bf16", True, True, True),
        # between two blocks of one token
        _residual_case("residual norm 1x4096", 1, 4096, "bf16", True, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv_step", "ssm", "ssm", "ssm_step", "gated", "residual"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    act = rng.choice(["silu", "silu", "none"])
    K = rng.choice([2, 3, 4, 4])
    some = lambda hi: _log(rng, 1, hi)  # noqa: E731
    if op == "conv":
        C = _log(rng, 16, 12288)
        T = _log(rng, 1, max(1, min(16384, 8192 * 12288 // (C * (2 if dtype == "f32" else 1)))))
        c = _conv_case("", T, some(16), C, K, dtype, act, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "conv_step":
        c = _conv_step_case("", some(256), _log(rng, 16, 12288), K, dtype, act, rng.random() < 0.5)
    elif op in ("ssm", "ssm_step"):
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.choice([1, 2, 3, 4])
        P, S = 16 * rng.randint(1, 8), rng.choice([16, 32, 64, 128])
        if op == "ssm":
            T = _log(rng, 1, 8192 if dtype == "bf16" else 4096)
            c = _ssm_case("", T, some(16), H, P, S, G, dtype, rng.random() < 0.5, rng.random() < 0.7)
        else:
            c = _ssm_step_case("", some(256), H, P, S, G, dtype, rng.random() < 0.7)
    elif op == "gated":
        H, D = rng.randint(1, 32), rng.choice([16, 64, 100, 128, rng.randint(1, 512)])
        c = _gated_case("", _log(rng, 1, max(1, min(8192, 8192 * 32 * 64 // (H * D)))), H, D, dtype,
                        rng.choice(["silu", "sigmoid"]), rng.random() < 0.5, rng.random() < 0.5)
    else:
        C = _log(rng, 16, 8192)
        c = _residual_case("", _log(rng, 1, min(16384, 8192 * 2048 // C)), C, dtype, rng.random() < 0.5,
                           rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ---- what a program has in hand ---------------------------------------------------

def _bounds(c):
    """First tokens of the N sequences and the end of the last: T tokens cut at random places."""
    T, N = c["T"], c["N"]
    rng = random.Random(T * 1009 + N)
    return [0] + sorted(rng.randint(0, T) for _ in range(N - 1)) + [T]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = TYPES[c["dtype"]]
    rand = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    uniform = lambda *s: torch.rand(*s, generator=gen, device=DEV)  # noqa: E731
    s = {"case": c}
    if "T" in c and "N" in c:
        s["bounds"] = _bounds(c)
        s["cu"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
    if c["op"] in ("conv", "conv_step"):
        C, K, N = c["C"], c["K"], c["N"]
        s["x"] = rand(c.get("T", N), C).to(dt)
        s["weight"] = (2 * uniform(C, K) - 1) / math.sqrt(K)
        s["bias"] = 0.1 * rand(C) if c["bias"] else None
        s["state"] = rand(N, K - 1, C).to(dt) if c["op"] == "conv_step" or c["cached"] else None
    elif c["op"] in ("ssm", "ssm_step"):
        H, P, S, G, N = c["H"], c["P"], c["S"], c["G"], c["N"]
        T = c.get("T", N)
        # x, B and C are parts of one convolved row; steps that forget little, as such layers are initialised
        row = rand(T, H * P + 2 * G * S)
        row = (row * torch.sigmoid(row)).to(dt)
        s["x"] = row[:, :H * P].unflatten(1, (H, P))
        s["b"] = row[:, H * P:H * P + G * S].unflatten(1, (G, S))
        s["c"] = row[:, H * P + G * S:].unflatten(1, (G, S))
        s["dt"] = 0.5 * rand(T, H)
        step = torch.exp(math.log(1e-3) + uniform(H) * math.log(100.0))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["a"] = -(1 + 15 * uniform(H))
        s["skip"] = 1 + 0.1 * rand(H) if c["skip"] else None
        s["state"] = 0.1 * rand(N, H, S, P) if c["op"] == "ssm_step" or c["cached"] else None
    elif c["op"] == "gated":
        T, H, D = c["T"], c["H"], c["D"]
        s["x"], s["gate"] = rand(T, H, D).to(dt), rand(T, H, D).to(dt)
        s["weight"] = 1 + 0.1 * rand(*((D,) if c["shared"] else (H, D)))
    else:
        T, C = c["T"], c["C"]
        s["x"], s["residual"] = (0.5 * rand(T, C)).to(dt), (3 * rand(T, C)).to(dt)
        s["weight"] = 1 + 0.1 * rand(C)
        s["post"] = 1 + 0.1 * rand(C) if c["post"] else None
        s["gate"] = rand(T, C).to(dt) if c["gate"] else None
        s["scale"] = uniform(C) if c["scale"] else None
    if own:
        from gated_delta_rule_109_amd import kda
        s["act"] = {"none": kda.ACT_NONE, "silu": kda.ACT_SILU, "sigmoid": kda.ACT_SIGMOID}[c.get("act", "none")]
        if c["op"] == "ssm":
            s["workspace"] = kda.ssm_workspace(c["N"], c["T"], c["H"], c["S"], c["P"], DEV)
    return s


# ---- plain forms --------------------------------------------------------------------

def _act(x, act):
    if act == "none":
        return x
    y = 1.0 / (1.0 + torch.exp(-x))
    return x * y if act == "silu" else y


def _conv_rows(s, c, rows):
    """Rows (state and inputs of one sequence or of one step, [.., K - 1 + L, C]) to outputs [.., L, C]."""
    K = c["K"]
    L = rows.shape[-2] - K + 1
    y = sum(rows[..., j:j + L, :] * s["weight"][:, j] for j in range(K))
    if s["bias"] is not None:
        y = y + s["bias"]
    return _act(y, c["act"]).to(s["x"].dtype)


def _conv(s, c):
    x, K = s["x"], c["K"]
    ys, ends = [], []
    for n, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        before = s["state"][n] if s["state"] is not None else x.new_zeros(K - 1, c["C"])
        rows = torch.cat([before, x[a:b]])
        ys.append(_conv_rows(s, c, rows.float()))
        ends.append(rows[b - a:])
    return {"y": torch.cat(ys), "state": torch.stack(ends)}


def _conv_step(s, c):
    rows = torch.cat([s["state"], s["x"][:, None]], 1)
    y = _conv_rows(s, c, rows.float())[:, 0]
    s["state"].copy_(rows[:, 1:])
    return {"y": y, "state": s["state"]}


def _delta(s):
    """Step sizes: softplus of the logits with their bias."""
    v = s["dt"] + s["dt_bias"]
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _heads(v, H):
    """Groups [.., G, S] in fp32, repeated for their heads."""
    return v.float().repeat_interleave(H // v.shape[-2], dim=-2)


def _ssm_sequence(s, c, x, delta, b, cc, state):
    """One sequence (x [L, H, P] fp32): the chunked form. Sums of decay logarithms in 64 bits."""
    L, H, P = x.shape
    S = b.shape[-1]
    n = -(-L // CHUNK)
    pad = n * CHUNK - L

    def chunks(v):          # [L, H, ..] -> [n, H, CHUNK, ..], zeros behind the end
        v = torch.cat([v, v.new_zeros(pad, *v.shape[1:])]) if pad else v
        return v.reshape(n, CHUNK, *v.shape[1:]).transpose(1, 2).contiguous()

    X, B, Cc, d = chunks(x), chunks(b), chunks(cc), chunks(delta)
    cum = (d.double() * s["a"].double()[:, None]).cumsum(-1)                       # [n, H, CHUNK]
    later = torch.ones(CHUNK, CHUNK, device=DEV, dtype=torch.bool).tril()
    decay = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~later, -math.inf)).float()
    y = (Cc @ B.transpose(-1, -2) * decay * d[..., None, :]) @ X
    left = torch.exp(cum[..., -1:] - cum).float() * d
    local = (B * left[..., None]).transpose(-1, -2).contiguous() @ X               # [n, H, S, P]
    whole = torch.exp(cum[..., -1]).float()
    before = torch.empty(n, H, S, P, device=DEV)
    for i in range(n):
        before[i] = state
        state = whole[i, :, None, None] * state + local[i]
    y = y + torch.exp(cum).float()[..., None] * (Cc @ before)
    return y.transpose(1, 2).reshape(n * CHUNK, H, P)[:L], state


def _ssm(s, c):
    H, P, S = c["H"], c["P"], c["S"]
    x, delta = s["x"].float(), _delta(s)
    b, cc = _heads(s["b"], H), _heads(s["c"], H)
    ys, ends = [], []
    for n, (i, j) in enumerate(zip(s["bounds"], s["bounds"][1:])):
        state = s["state"][n] if s["state"] is not None else torch.zeros(H, S, P, device=DEV)
        if j > i:
            y, state = _ssm_sequence(s, c, x[i:j], delta[i:j], b[i:j], cc[i:j], state)
            ys.append(y)
        ends.append(state)
    y = torch.cat(ys)
    if s["skip"] is not None:
        y = y + s["skip"][:, None] * x
    return {"y": y.to(s["x"].dtype), "state": torch.stack(ends)}


def _ssm_step(s, c):
    H = c["H"]
    x, delta = s["x"].float(), _delta(s)
    b, cc = _heads(s["b"], H), _heads(s["c"], H)
    alpha = torch.exp(delta * s["a"])
    s["state"].mul_(alpha[..., None, None]).add_((delta[..., None] * b)[..., None] * x[..., None, :])
    y = (s["state"] * cc[..., None]).sum(-2)
    if s["skip"] is not None:
        y = y + s["skip"][:, None] * x
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _norm(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _gated(s, c):
    x, g = s["x"].float(), _act(s["gate"].float(), c["act"])
    y = _norm(x * g) * s["weight"] if c["gate_first"] else _norm(x) * s["weight"] * g
    return y.to(s["x"].dtype)


def _residual(s, c):
    x = s["x"].float()
    if s["post"] is not None:
        x = _norm(x) * s["post"]
    if s["gate"] is not None:
        x = x * _act(s["gate"].float(), "sigmoid")
    if s["scale"] is not None:
        x = x * s["scale"]
    r = s["residual"].float() + 0.5 * x
    return {"residual": r.to(s["x"].dtype), "y": (_norm(r) * s["weight"]).to(s["x"].dtype)}


_PLAIN = {"conv": _conv, "conv_step": _conv_step, "ssm": _ssm, "ssm_step": _ssm_step, "gated": _gated,
          "residual": _residual}


def run(state):
    s, c = state, state["case"]
    return _run_own(s, c) if own else _PLAIN[c["op"]](s, c)


def _run_own(s, c):
    from gated_delta_rule_109_amd import kda
    op = c["op"]
    if op == "conv":
        y, end = kda.conv_prefill(s["x"], s["weight"], s["bias"], cu_seqlens=s["cu"], initial_state=s["state"],
                                  activation=s["act"])
        return {"y": y, "state": end}
    if op == "conv_step":
        return {"y": kda.conv_step(s["x"], s["weight"], s["state"], s["bias"], activation=s["act"]),
                "state": s["state"]}
    if op == "ssm":
        y, end = kda.ssm_prefill(s["x"], s["dt"], s["a"], s["b"], s["c"], skip=s["skip"], dt_bias=s["dt_bias"],
                                 dt_softplus=True, cu_seqlens=s["cu"], initial_state=s["state"],
                                 workspace=s["workspace"])
        return {"y": y, "state": end}
    if op == "ssm_step":
        return {"y": kda.ssm_step(s["x"], s["dt"], s["a"], s["b"], s["c"], s["state"], skip=s["skip"],
                                  dt_bias=s["dt_bias"], dt_softplus=True), "state": s["state"]}
    if op == "gated":
        return kda.gated_norm(s["x"], s["gate"], s["weight"], activation=s["act"], gate_first=c["gate_first"],
                              eps=1e-6)
    residual, y = kda.residual_norm(s["x"], s["residual"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                    activation=kda.ACT_SIGMOID, scale=s["scale"], alpha=0.5, eps=1e-6)
    return {"residual": residual, "y": y}


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("conv", "conv_step"):
        N, C, K = c["N"], c["C"], c["K"]
        T = c.get("T", N)
        states = 2 if c["op"] == "conv_step" or c["cached"] else 1
        return {"bytes": e * (2 * T * C + states * N * (K - 1) * C) + 4 * C * (K + c["bias"]),
                "flops": T * C * (2.0 * K + (4 if c["act"] == "silu" else 0))}
    if c["op"] in ("ssm", "ssm_step"):
        N, H, P, S, G = c["N"], c["H"], c["P"], c["S"], c["G"]
        T = c.get("T", N)
        states = 2 if c["op"] == "ssm_step" or c["cached"] else 1
        return {"bytes": T * (2 * e * H * P + 2 * e * G * S + 4 * H) + 4 * states * N * H * P * S,
                "flops": 5.0 * T * H * P * S}
    if c["op"] == "gated":
        return {"bytes": 3 * e * c["T"] * c["H"] * c["D"], "flops": 9.0 * c["T"] * c["H"] * c["D"]}
    arrays = 5 if c["gate"] else 4
    return {"bytes": arrays * e * c["T"] * c["C"] + 4 * c["C"] * (1 + c["post"] + c["scale"]),
            "flops": 10.0 * c["T"] * c["C"]}


# ---- exact values: the definitions in 64 bits, token by token -----------------------------

def _exact_act(v, act):
    return v if act == "none" else torch.sigmoid(v) * (v if act == "silu" else 1.0)


def _exact_conv(s, c):
    K, C = c["K"], c["C"]
    steps = c["op"] == "conv_step"
    bounds = list(range(c["N"] + 1)) if steps else s["bounds"]
    x = s["x"].double()
    out = torch.zeros_like(x) + (s["bias"].double() if s["bias"] is not None else 0.0)
    first = torch.zeros(x.shape[0], dtype=torch.long, device=DEV)
    owner = torch.zeros(x.shape[0], dtype=torch.long, device=DEV)
    for n, (a, b) in enumerate(zip(bounds, bounds[1:])):
        first[a:b], owner[a:b] = a, n
    at = torch.arange(x.shape[0], device=DEV)
    past = s["state"].double() if s["state"] is not None else x.new_zeros(c["N"], K - 1, C)
    for j in range(K):          # tap j looks K - 1 - j tokens back
        src = at - (K - 1 - j)
        row = torch.where((src >= first)[:, None], x[src.clamp(min=0)],
                          past[owner, (src - first + K - 1).clamp(0, K - 2)])
        out += s["weight"][:, j].double() * row
    ends = []
    for n, (a, b) in enumerate(zip(bounds, bounds[1:])):
        row = lambda i: x[i] if i >= a else past[n, K - 1 + i - a]  # noqa: E731
        ends.append(torch.stack([row(i) for i in range(b - K + 1, b)]))
    return {"y": _exact_act(out, c["act"]), "state": torch.stack(ends)}


def _exact_ssm(s, c):
    H, P, S, N = c["H"], c["P"], c["S"], c["N"]
    bounds = list(range(N + 1)) if c["op"] == "ssm_step" else s["bounds"]
    x = s["x"].double()
    per = H // c["G"]
    group = torch.arange(H, device=DEV) // per
    b, cc = s["b"].double()[:, group], s["c"].double()[:, group]
    delta = torch.logaddexp(torch.zeros((), device=DEV, dtype=torch.float64), s["dt"].double() + s["dt_bias"].double())
    alpha = torch.exp(delta * s["a"].double())
    xd = delta[..., None] * x
    state = s["state"].double().clone() if s["state"] is not None else x.new_zeros(N, H, S, P)
    y = torch.zeros_like(x)
    starts = torch.tensor(bounds[:-1], device=DEV)
    lengths = [j - i for i, j in zip(bounds, bounds[1:])]
    order = sorted(range(N), key=lambda n: -lengths[n])      # longest first: the live ones are a prefix
    state = state[torch.tensor(order, device=DEV)]
    starts = starts[torch.tensor(order, device=DEV)]
    live = N
    for t in range(max(lengths)):
        while lengths[order[live - 1]] <= t:
            live -= 1
        i = starts[:live] + t
        st = state[:live]
        st.mul_(alpha[i][..., None, None])
        st.add_(b[i][..., None] * xd[i][..., None, :])
        y[i] = torch.matmul(cc[i][..., None, :], st)[..., 0, :]
    if s["skip"] is not None:
        y += s["skip"].double()[:, None] * x
    back = torch.empty_like(state)
    back[torch.tensor(order, device=DEV)] = state
    return {"y": y, "state": back}


def _exact_gated(s, c):
    x, z, w = s["x"].double(), s["gate"].double(), s["weight"].double()
    g = _exact_act(z, c["act"])
    v = x * g if c["gate_first"] else x
    y = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6) * w
    return y if c["gate_first"] else y * g


def _exact_residual(s, c):
    C = c["C"]
    v = s["x"].double()
    if c["post"]:
        v = s["post"].double() * v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / C + 1e-6)
    if c["gate"]:
        v = v * torch.sigmoid(s["gate"].double())
    if c["scale"]:
        v = v * s["scale"].double()
    r = s["residual"].double() + 0.5 * v
    return {"residual": r, "y": s["weight"].double() * r / torch.sqrt(r.pow(2).sum(-1, keepdim=True) / C + 1e-6)}


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"conv": _exact_conv, "conv_step": _exact_conv, "ssm": _exact_ssm, "ssm_step": _exact_ssm,
            "gated": _exact_gated, "residual": _exact_residual}[c["op"]](s, c)
