"""The speculative step (tree attention over the state, draft verification,
path commit) and the 8-bit state cache on the GPU, against the fp64 oracle.

Tolerances:
  tree outputs   element by element: the oracle's error bound for the arithmetic
                 (oracle.speculative.tree_bound; fp32 products, or two-term bf16
                 operands of 3 * 2^-18 relative error each for bf16 tensors) plus,
                 for bf16 outputs, the rounding to bf16, 2^-8 |o|
  committed states  a step rounds its sums of D terms and a few products, at most
                 (D + 16) 2^-24 of the sizes involved; for unit keys and write
                 strengths in [0, 1] a step does not enlarge a column's error
                 (I - b k k^T and the decays have norm <= 1), so over a path of L
                 tokens a column is at most L (D + 16) 2^-24 (|S column| + |d|) off
  verification and cache   equal
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_109_amd import kda
from gated_delta_rule_109_amd.workloads import make_inputs
from oracle import frontend, speculative

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LN_HALF = float(np.log(0.5))
BF16, F32 = torch.bfloat16, torch.float32
# relative error of one product of the unrolled form, by the tensors' type
PRODUCT = {BF16: 3 * 3 * 2.0 ** -18, F32: 0.0}
# hardware rcp, rsqrt and exp2 of the front end: a few units of 2^-23 on each input
FRONT_END = 16 * 2.0 ** -23


def dev(a, dt=F32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dt).to(DEV)


def host(x):
    return x.float().cpu().numpy()


def random_parents(N, T, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "chain":
        return np.tile(np.arange(T) - 1, (N, 1)).astype(np.int32)
    if kind == "star":
        return np.tile(np.minimum(np.arange(T), 1) - 1, (N, 1)).astype(np.int32)
    p = np.array([[-1] + [int(rng.integers(0, i)) for i in range(1, T)] for _ in range(N)], np.int32)
    if kind == "forest":
        p[rng.random((N, T)) < 0.3] = -1
    if kind == "bad":          # values that count as -1
        for n in range(N):
            for i in range(T):
                p[n, i] = rng.choice([p[n, i], -7, i, T + 3, 2 ** 31 - 1, -2 ** 31])
    return p


class Step:
    """Inputs of a step on the host (values as the device holds them) and on the device."""

    def __init__(self, N, T, H, D, dtype, seed, gate=kda.GATE_CHANNEL, flags=0, g_min=LN_HALF):
        raw = flags != 0
        inp = make_inputs(N * T, H, D, seed=seed, lengths=[T] * N, initial_state=True, bf16=dtype is BF16, raw=raw)
        self.s0 = inp.initial_state
        q, k, v, g, b = (x.reshape(N, T, *x.shape[1:]) for x in (inp.q, inp.k, inp.v, inp.g, inp.beta))
        if g_min != LN_HALF and not raw:
            g = (g * np.float32(g_min / LN_HALF)).astype(np.float32)
        if gate == kda.GATE_HEAD:
            g = np.ascontiguousarray(g[..., 0])
        elif gate == kda.GATE_NONE:
            g = None
        self.args = [dev(q, dtype), dev(k, dtype), dev(v, dtype), dev(g), dev(b)]
        if raw:
            z = np.zeros((N, T, H)) if g is None else g
            q, k, z, b = frontend.apply(q, k, z, b, flags, 1e-6)
            g = None if g is None else z
        self.q, self.k, self.v, self.g, self.b = q, k, v, g, b
        self.state = dev(self.s0)
        self.g_min = g_min
        self.product = PRODUCT[dtype] + (FRONT_END if raw else 0.0)
        self.options = kda.Options(flags=flags, gate=gate) if raw or gate != kda.GATE_CHANNEL else None

    def check_tree(self, o, parents, num_nodes=None, scale=1.0):
        ref = speculative.decode_tree(self.q, self.k, self.v, self.g, self.b, self.s0, parents, num_nodes, scale,
                                      self.g_min)
        N, T = ref.shape[:2]
        out = host(o)
        for n in range(N):
            nt = T if num_nodes is None else int(np.clip(num_nodes[n], 0, T))
            par = speculative.parents_of(None if parents is None else parents[n], T)
            tol = speculative.tree_bound(self.q[n], self.k[n], self.v[n], None if self.g is None else self.g[n],
                                         self.b[n], self.s0[n], par, nt, scale, self.g_min, self.product)
            if o.dtype is BF16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref[n, :nt])
            err = np.abs(out[n, :nt] - ref[n, :nt])
            assert (err <= tol).all(), f"sequence {n}: {np.nanmax(err / tol):.2f} of the tolerance"


TREES = [
    # N, T, H, D, dtype, tree, gate, flags, g_min
    (1, 1, 1, 128, BF16, "chain", 0, 0, LN_HALF),
    (2, 8, 3, 128, BF16, "bushy", 0, 0, LN_HALF),
    (3, 16, 2, 128, BF16, "bushy", 0, 0, LN_HALF),
    (2, 17, 2, 128, BF16, "chain", 0, 0, LN_HALF),
    (2, 31, 1, 128, F32, "forest", 0, 0, LN_HALF),
    (1, 33, 2, 128, F32, "bushy", 1, 0, LN_HALF),
    (1, 48, 1, 128, BF16, "star", 2, 0, LN_HALF),
    (1, 64, 2, 128, BF16, "bushy", 0, kda.FE_ALL, LN_HALF),
    (1, 64, 1, 128, BF16, "chain", 0, 0, LN_HALF),
    (1, 64, 1, 128, F32, "chain", 0, 0, LN_HALF),
    (2, 16, 2, 128, F32, "bushy", 0, kda.FE_ALL, LN_HALF),
    (2, 12, 2, 128, BF16, "bad", 1, kda.FE_ALL, LN_HALF),
    (1, 64, 2, 128, BF16, "chain", 0, 0, -5.0),
    (2, 5, 1, 128, F32, "chain", 0, 0, -40.0),
    (1, 20, 1, 128, BF16, "bushy", 0, kda.FE_ALL, -1e30),
    (3, 1, 2, 16, F32, "chain", 0, 0, LN_HALF),
    (2, 23, 3, 16, BF16, "bushy", 0, 0, LN_HALF),
    (1, 64, 2, 16, F32, "chain", 0, kda.FE_ALL, -5.0),
    (1, 64, 2, 16, BF16, "bad", 2, kda.FE_L2NORM_QK | kda.FE_BETA_LOGITS, LN_HALF),
]


@pytest.mark.parametrize("N,T,H,D,dtype,tree,gate,flags,g_min", TREES)
def test_tree(N, T, H, D, dtype, tree, gate, flags, g_min):
    s = Step(N, T, H, D, dtype, 100 + T, gate, flags, g_min)
    par = random_parents(N, T, tree, T)
    before = s.state.clone()
    o = kda.decode_tree(*s.args, s.state, dev(par, torch.int32), scale=0.7, g_min=g_min, options=s.options)
    s.check_tree(o, par, scale=0.7)
    assert torch.equal(s.state, before)
    if tree == "chain":
        assert torch.equal(o, kda.decode_tree(*s.args, s.state, None, scale=0.7, g_min=g_min, options=s.options))


@pytest.mark.parametrize("N,T,H,D,dtype,tree,gate,flags,g_min", [x for x in TREES if x[4] is BF16])
def test_tree_of_bf16_within_the_bound_of_fp32_products(N, T, H, D, dtype, tree, gate, flags, g_min):
    """bf16 tensors against the bound of fp32 arithmetic, without the allowance
    for operands of two bf16 terms, and the one rounding of the outputs."""
    s = Step(N, T, H, D, dtype, 900 + T, gate, flags, g_min)
    s.product = FRONT_END if flags else 0.0
    par = random_parents(N, T, tree, T + 1)
    o = kda.decode_tree(*s.args, s.state, dev(par, torch.int32), scale=1.3, g_min=g_min, options=s.options)
    s.check_tree(o, par, scale=1.3)


@pytest.mark.parametrize("T,D,dtype", [(16, 128, BF16), (40, 128, F32), (16, 128, F32), (64, 128, BF16), (19, 16, BF16)])
def test_tree_of_each_sequences_own_size(T, D, dtype):
    nodes = np.array([0, 1, T, T + 9, -3, T // 2], np.int32)
    N, H = len(nodes), 2
    s = Step(N, T, H, D, dtype, 7)
    par = random_parents(N, T, "bushy", 3)
    # what lies behind a sequence's last node is never read
    live = torch.arange(T, device=DEV) < dev(nodes, torch.int32)[:, None]
    for x in s.args:
        x[~live] = float("nan")
    o = torch.full((N, T, H, D), 42.0, device=DEV, dtype=dtype)
    kda.decode_tree(*s.args, s.state, dev(par, torch.int32), dev(nodes, torch.int32), o=o)
    s.check_tree(o, par, nodes)
    assert (o[~live] == 42.0).all()


@pytest.mark.parametrize("T,D,dtype,g_min", [(16, 128, BF16, LN_HALF), (50, 128, BF16, LN_HALF), (21, 128, F32, LN_HALF),
                                             (16, 16, F32, LN_HALF), (50, 128, BF16, -5.0), (20, 128, F32, -5.0),
                                             (50, 16, BF16, -5.0), (9, 128, F32, -100.0)])
@pytest.mark.parametrize("what", ["v", "k", "q", "beta"])
def test_a_nodes_nan_reaches_its_descendants_only(T, D, dtype, g_min, what):
    s = Step(1, T, 2, D, dtype, 21, g_min=g_min)
    par = random_parents(1, T, "bushy", 8)
    p = dev(par, torch.int32)
    clean = kda.decode_tree(*s.args, s.state, p, g_min=g_min)
    i = 3
    x = s.args[["q", "k", "v", "g", "beta"].index(what)]
    if what == "beta":
        x[0, i, 1] = float("inf")
    else:
        x[0, i, 1, 5] = float("nan")
    o = kda.decode_tree(*s.args, s.state, p, g_min=g_min)
    below = {i}
    for t in range(i + 1, T):
        if int(par[0, t]) in below:
            below.add(t)
    hit = torch.zeros(1, T, 2, dtype=torch.bool, device=DEV)
    hit[0, [i] if what == "q" else sorted(below), 1] = True
    assert torch.equal(o[~hit], clean[~hit])
    bad = ~torch.isfinite(o[hit])
    # a value's NaN stays in its column, the others reach every one
    assert bad[:, 5].all() if what == "v" else bad.all()
    if what == "v":
        rest = torch.ones(D, dtype=torch.bool, device=DEV)
        rest[5] = False
        assert torch.equal(o[hit][:, rest], clean[hit][:, rest])


@pytest.mark.parametrize("gate,flags", [(kda.GATE_CHANNEL, 0), (kda.GATE_HEAD, 0), (kda.GATE_CHANNEL, kda.FE_ALL)])
@pytest.mark.parametrize("T,D,dtype,g_min", [(16, 128, BF16, LN_HALF), (50, 128, BF16, LN_HALF), (21, 128, F32, LN_HALF),
                                             (16, 16, F32, LN_HALF), (50, 128, BF16, -5.0), (20, 128, F32, -5.0),
                                             (50, 16, BF16, -5.0), (9, 128, F32, -100.0)])
def test_a_nan_decay_reaches_its_nodes_descendants_only(T, D, dtype, g_min, gate, flags):
    """A NaN log-decay (or logit) makes every column of its node and the nodes
    below it NaN, the state of a path through it too; infinite ones are clamped."""
    s = Step(2, T, 2, D, dtype, 22, gate, flags, g_min)
    par = random_parents(2, T, "bushy", 8)
    p, opts = dev(par, torch.int32), dict(g_min=g_min, options=s.options)
    g = s.args[3]
    i, h = 3, 1
    g[1, i, h].reshape(-1)[-1] = float("nan")
    # behind a sequence's last node nothing is read, a NaN decay neither
    nodes = np.array([T - 2, T], np.int32)
    g[0, T - 2:] = float("nan")
    o = kda.decode_tree(*s.args, s.state, p, dev(nodes, torch.int32), **opts)
    hit = torch.zeros(2, T, 2, dtype=torch.bool, device=DEV)
    below = {i}
    for t in range(i + 1, T):
        if int(par[1, t]) in below:
            below.add(t)
    hit[1, sorted(below), h] = True
    live = torch.arange(T, device=DEV) < dev(nodes, torch.int32)[:, None]
    assert torch.isnan(o[hit]).all()
    # the other nodes against the oracle, which has the inputs without NaN (not bit
    # for bit against a run without: the decays' reference in a block of nodes, and
    # so the rounding, goes by the decays of all its live nodes)
    ref = speculative.decode_tree(s.q, s.k, s.v, s.g, s.b, s.s0, par, nodes, 1.0, g_min)
    for n in range(2):
        rows = (~hit & live[..., None])[n, :nodes[n]].cpu().numpy()
        tol = speculative.tree_bound(s.q[n], s.k[n], s.v[n], s.g[n], s.b[n], s.s0[n],
                                     speculative.parents_of(par[n], T), nodes[n], 1.0, g_min, s.product)
        if dtype is BF16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref[n, :nodes[n]])
        assert (np.abs(host(o[n, :nodes[n]]) - ref[n, :nodes[n]]) <= tol)[rows].all()
    # the commit of a path through the node, and of one beside it
    path = torch.full((2, T), -1, device=DEV, dtype=torch.int32)
    path[0, :2], path[1, :2] = torch.tensor([0, 1]), torch.tensor([0, i])
    state = s.state.clone()
    kda.commit_path(*s.args[1:], state, path, torch.full((2,), 2, device=DEV, dtype=torch.int32), **opts)
    assert torch.isfinite(state[0]).all() and torch.isfinite(state[1, 0]).all() and torch.isnan(state[1, 1]).all()
    # infinities: the floor and no decay (as logits the other way round)
    ends = [s.args[3].clone() for _ in range(2)]
    low, none = (float("-inf"), float("inf")) if not flags else (float("inf"), float("-inf"))
    for x, inf, stand_in in ((ends[0], low, 1e30 if flags else -1e30), (ends[1], none, -1e30 if flags else 1e30)):
        x.nan_to_num_(nan=0.25)
        y = x.clone()
        x[1, i], y[1, i] = inf, stand_in
        both = [kda.decode_tree(*s.args[:3], z, s.args[4], s.state, p, **opts) for z in (x, y)]
        assert torch.equal(*both) and torch.isfinite(both[0]).all()


@pytest.mark.parametrize("T,D,dtype,g_min", [(16, 128, BF16, LN_HALF), (30, 128, BF16, LN_HALF), (50, 128, BF16, LN_HALF),
                                             (50, 128, BF16, -5.0), (50, 128, F32, LN_HALF), (20, 16, BF16, LN_HALF),
                                             (9, 128, BF16, -100.0)])
def test_a_nodes_finite_values_near_the_largest_stay_its_own(T, D, dtype, g_min):
    """A delta row of 3.4014e38, which is finite in fp32 (the largest: 3.4028e38)
    but rounds to infinity in bf16, belongs to its node and descendants only."""
    s = Step(1, T, 1, D, dtype, 77, g_min=g_min)
    par = random_parents(1, T, "bushy", 8)
    p = dev(par, torch.int32)
    i = 3
    k, v, g, b = s.args[1:]
    s.state[0, 0, 2] = -1.2e36
    k[0, i] = 0.0
    k[0, i, 0, 2] = 1.0
    g[0, :, 0, 2] = 0.0                                       # S^T (E k) = -1.2e36 at node i
    b[0, i] = 1.0
    # the other nodes neither read nor write that channel
    for x in s.args[:2]:
        x[0, [t for t in range(T) if t != i], 0, 2] = 0.0
    clean = kda.decode_tree(*s.args, s.state, p, g_min=g_min)
    v[0, i] = torch.finfo(BF16).max                           # 3.3895e38, and 1.2e36 from the state
    o = kda.decode_tree(*s.args, s.state, p, g_min=g_min)
    below = {i}
    for t in range(i + 1, T):
        if int(par[0, t]) in below:
            below.add(t)
    rest = [t for t in range(T) if t not in below]
    assert len(rest) > 4 and torch.isfinite(clean[0, rest]).all()
    assert torch.equal(o[0, rest], clean[0, rest])


@pytest.mark.parametrize("D,dtype", [(128, BF16), (128, F32), (16, BF16), (16, F32)])
@pytest.mark.parametrize("T,g_min,flags,gate", [(64, -5.0, 0, 0), (40, -5.0, kda.FE_ALL, 0), (33, -2.5, 0, 1), (16, -5.0, 0, 0),
                                                (48, -12.0, 0, 0), (64, -80.0, 0, 0)])
def test_deep_trees(T, D, dtype, g_min, flags, gate):
    """Decays that span more than fp32: chains, bushy trees, and branches that
    mix deep and shallow nodes in one block (which no block's reference fits),
    as sequences of one call."""
    N, H = 5, 1
    s = Step(N, T, H, D, dtype, 31 + T, gate, flags, g_min)
    par = random_parents(N, T, "bushy", T)
    par[0] = np.arange(T) - 1
    par[1] = np.maximum(np.arange(T) - 2, -1)                # two chains, in turn
    par[2] = np.arange(T) - 1
    par[2, T // 2::3] = 0                                    # branches off the root beside the deep chain
    nodes = np.array([T, T, T, T, T - 3], np.int32)
    o = kda.decode_tree(*s.args, s.state, dev(par, torch.int32), dev(nodes, torch.int32), g_min=g_min, options=s.options)
    s.check_tree(o, par, nodes)
    assert torch.equal(o, kda.decode_tree(*s.args, s.state, dev(par, torch.int32), dev(nodes, torch.int32), g_min=g_min,
                                          options=s.options))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tree_of_very_many_heads(dtype):
    """A row of all heads past 2^24 bytes (another kernel) against the same
    memory as two sequences of half the heads."""
    H, D = 32768, 128
    gen = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (torch.randn(1, 1, H, D, device=DEV, generator=gen) for _ in range(3))
    q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    q, k, v = (x.to(dtype) for x in (q, k, v))
    g = -torch.rand(1, 1, H, D, device=DEV, generator=gen)
    b = torch.rand(1, 1, H, device=DEV, generator=gen)
    st = 0.1 * torch.randn(1, H, D, D, device=DEV, generator=gen)
    two = lambda x: x.reshape(2, -1, H // 2, *x.shape[3:])  # noqa: E731
    o = kda.decode_tree(q, k, v, g, b, st).reshape(2, 1, H // 2, D)
    ref = kda.decode_tree(*(two(x) for x in (q, k, v, g)), two(b), st.reshape(2, H // 2, D, D))
    # one node: o = (E q) S + (q . k) d, terms below |q||S| + |d| < 8; both sides
    # within (D + 22) 2^-24 (plus the operand splits) of it and a rounding of o
    tol = 2 * 8 * (150 * 2.0 ** -24 + PRODUCT[dtype])
    err = (o.float() - ref.float()).abs()
    assert (err <= tol + (2.0 ** -7 if dtype is BF16 else 0.0) * ref.float().abs()).all()


@pytest.mark.parametrize("D,dtype", [(128, BF16), (128, F32), (16, BF16)])
@pytest.mark.parametrize("T,g_min", [(1, LN_HALF), (16, LN_HALF), (30, LN_HALF), (45, LN_HALF), (64, LN_HALF),
                                     (64, -5.0), (20, -5.0), (7, -100.0)])
def test_operands_keep_fp32s_digits(T, D, dtype, g_min):
    """Sums that cancel down to digits 2^-20 below their terms. Every product and
    every sum here is exact in fp32, in any order (multiples of 2^-20 below 4), so
    the outputs are too; operands of fewer than 21 bits would lose them."""
    m = torch.arange(1, D + 1, device=DEV).float() * 2.0 ** -20     # (at most 8 bits: exact in bf16)
    state = torch.zeros(2, 1, D, D, device=DEV)
    state[:, 0, 2] = 1.0 + 2.0 ** -9 + m
    state[:, 0, 5] = 1.0 + 2.0 ** -9
    q = torch.zeros(2, T, 1, D, device=DEV, dtype=dtype)
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    g = torch.zeros(2, T, 1, D, device=DEV)
    beta = torch.zeros(2, T, 1, device=DEV)
    # sequence 0 reads q = e_2 - e_5 from the state: m
    q[0, :, 0, 2], q[0, :, 0, 5] = 1.0, -1.0
    # sequence 1: the last node writes d = v - S^T k with k = e_2 - e_5 and reads what it wrote: -m + v
    k[1, T - 1, 0, 2], k[1, T - 1, 0, 5] = 1.0, -1.0
    beta[1, T - 1] = 1.0
    q[1, T - 1, 0, 5] = -1.0                                        # S^T q - d (k . e_5) = -S_5 + d
    v[1, T - 1] = 1.0
    o = kda.decode_tree(q, k, v, g, beta, state, g_min=g_min).double()
    assert torch.equal(o[0, :, 0], m.double().expand(T, D))
    # -S_5 + (1 - m) = -2^-9 - m: at most 12 bits, rounded to the outputs' type
    assert torch.equal(o[1, T - 1, 0], (-(2.0 ** -9) - m).to(dtype).double())


def test_tree_of_a_chain_is_the_token_decode():
    """The tree's outputs of a chain against kda_decode_tokens, which runs the
    recurrence: both within their bounds of the exact value, so within twice."""
    s = Step(3, 16, 2, 128, F32, 9)
    o = kda.decode_tree(*s.args, s.state, None)
    ref = kda.decode_tokens(*s.args, s.state.clone())
    s.check_tree(o, None)
    s.check_tree(ref, None)


@pytest.mark.parametrize("N,T,H,D,dtype,gate,flags,g_min", [
    (3, 1, 2, 128, BF16, 0, 0, LN_HALF), (4, 16, 2, 128, BF16, 0, 0, LN_HALF), (2, 64, 1, 128, F32, 0, 0, LN_HALF),
    (5, 23, 2, 128, F32, 1, 0, -5.0), (3, 9, 2, 128, BF16, 2, kda.FE_L2NORM_QK | kda.FE_BETA_LOGITS, LN_HALF),
    (3, 12, 1, 128, BF16, 0, kda.FE_ALL, -1e30), (4, 8, 3, 16, F32, 0, 0, LN_HALF), (3, 40, 2, 16, BF16, 0, kda.FE_ALL, LN_HALF),
])
def test_commit(N, T, H, D, dtype, gate, flags, g_min):
    s = Step(N, T, H, D, dtype, 300 + T, gate, flags, g_min)
    rng = np.random.default_rng(T)
    accept = rng.integers(0, T + 1, N).astype(np.int32)
    accept[0] = 0
    accept[-1] = T + 5                                       # counts as T
    path = rng.integers(0, T, (N, T)).astype(np.int32)       # any order, with repeats
    if N > 2:
        path[1, T // 2:] = -1                                # ends the path
        path[2, T - 1] = T
    out = kda.commit_path(*s.args[1:], s.state, dev(path, torch.int32), dev(accept, torch.int32), g_min=g_min,
                          options=s.options)
    assert out is s.state
    ref, size, lengths = speculative.commit_path(s.k, s.v, s.g, s.b, s.s0, path, accept, g_min)
    tol = lengths[:, None, None] * ((D + 16) * 2.0 ** -24 + (FRONT_END if flags else 0)) * size
    err = np.sqrt(((host(s.state) - ref) ** 2).sum(-2))
    assert (err <= tol).all(), f"{np.nanmax(err / np.maximum(tol, 1e-30)):.2f} of the tolerance"
    assert torch.equal(s.state[0], dev(s.s0)[0])             # bit for bit
    assert lengths[0] == 0


def test_commit_reads_listed_nodes_only():
    s = Step(2, 6, 2, 128, BF16, 5)
    path, accept = np.array([[0, 3, 5, -1, -1, -1]] * 2, np.int32), np.array([3, 2], np.int32)
    want = kda.commit_path(*s.args[1:], s.state.clone(), dev(path, torch.int32), dev(accept, torch.int32))
    for x in s.args:
        x[:, [1, 2, 4]] = float("nan")
        x[1, 5] = float("nan")
    got = kda.commit_path(*s.args[1:], s.state, dev(path, torch.int32), dev(accept, torch.int32))
    assert torch.equal(got, want) and torch.isfinite(got).all()


def probabilities(rng, N, T, V, dtype, peak=3.0, drift=1.0):
    z = peak * rng.standard_normal((N, T, V))
    p = np.exp(z - z.max(-1, keepdims=True))
    z = z + drift * rng.standard_normal((N, T, V))
    q = np.exp(z - z.max(-1, keepdims=True))
    return [torch.from_numpy((x / x.sum(-1, keepdims=True)).astype(np.float32)).to(dtype) for x in (p, q)]


def check_verify(target, draft, tokens, u, parents, nodes=None, **more):
    got = kda.verify_drafts(target.to(DEV), None if draft is None else draft.to(DEV), dev(tokens, torch.int32), dev(u),
                            dev(parents, torch.int32), dev(nodes, torch.int32), **more)
    want = speculative.verify(target.float().numpy(), None if draft is None else draft.float().numpy(), tokens, u, parents,
                              nodes)
    for a, b, name in zip(got, want, ("accept", "path", "next_token")):
        assert a.cpu().numpy().tolist() == b.tolist(), name
    return want


VERIFY = [
    # N, T, V, dtype, tree, draft
    (1, 1, 1, F32, "chain", False), (3, 4, 7, BF16, "chain", True), (1, 5, 1024, F32, "chain", True),
    (5, 8, 1025, F32, "chain", True), (4, 6, 4099, BF16, "chain", False), (2, 9, 9001, BF16, "bushy", True),
    (6, 16, 2049, F32, "bushy", True), (3, 64, 1000, F32, "bushy", True), (3, 64, 501, BF16, "star", False),
    (2, 33, 5003, F32, "bushy", False), (70, 5, 4097, F32, "chain", True), (66, 7, 8209, BF16, "bushy", True),
    (65, 3, 65537, F32, "chain", True), (2, 3, 300001, BF16, "star", True), (4, 12, 777, F32, "forest", True),
    (4, 12, 777, F32, "bad", False),
    # either side of the sizes at which the library spreads the rows over the GPU
    (2, 3, 49152, F32, "chain", True), (2, 3, 49153, F32, "chain", True), (3, 4, 49155, BF16, "bushy", False),
    (2, 4, 65537, F32, "bushy", True), (33, 3, 65539, BF16, "star", True), (257, 2, 16385, F32, "chain", True),
    (160, 2, 49157, BF16, "chain", False), (1025, 2, 40, F32, "chain", True), (1025, 2, 40, BF16, "chain", False),
]


@pytest.mark.parametrize("N,T,V,dtype,tree,with_draft", VERIFY)
def test_verify(N, T, V, dtype, tree, with_draft):
    rng = np.random.default_rng(V + T)
    target, draft = probabilities(rng, N, T, V, dtype)
    par = random_parents(N, T, tree, V)
    tokens = np.zeros((N, T), np.int32)
    for n in range(N):
        for i in range(1, T):
            w = draft[n, max(0, min(int(par[n, i]), T - 1))].double().numpy()
            tokens[n, i] = rng.choice(V, p=w / w.sum())
    u = rng.random((N, T)).astype(np.float32)
    nodes = None if N == 1 else rng.integers(0, T + 1, N).astype(np.int32)
    acc, _, _ = check_verify(target, draft if with_draft else None, tokens, u, None if tree == "chain" else par, nodes)
    if N >= 65 and with_draft:
        assert len(set(acc.tolist())) > 2           # the drafts are taken to different depths
    # low uniforms accept more, and draw from the first tokens
    check_verify(target, draft if with_draft else None, tokens, u * 0.1, None if tree == "chain" else par, nodes)


def test_verify_edges():
    """u at the ends of its range and outside it, rows of one token, rows with no
    weight, residuals that are 0, tokens out of range, repeated siblings, and
    entries that are no probabilities."""
    T, V = 4, 5000
    star = np.array([[-1, 0, 0, 0]], np.int32)
    p = torch.zeros(1, T, V)
    p[0, :, 4999] = 1.0
    tok = np.array([[0, 4999, 1, 2]], np.int32)
    for u0 in (0.0, 0.5, np.float32(1 - 2.0 ** -24), 1.0, 7.0, -1.0, np.nan):
        u = np.array([[u0, 0.0, 0.0, 0.0]], np.float32)
        un = np.where(np.isnan(u), 0.0, u)                  # NaN draws as 0
        for draft in (None, p):
            got = check_verify(p, draft, tok, u if not np.isnan(u0) else un, star)
            assert got[0][0] == 2 and got[2][0] == 4999
    # no child of weight, draft equal to target: the residual is 0, the draw is from the target
    tok = np.array([[0, 1, 1, 1]], np.int32)
    u = np.full((1, T), 0.5, np.float32)
    for draft in (None, p):
        got = check_verify(p, draft, tok, u, star)
        assert got[0][0] == 1 and got[2][0] == 4999
    # without draft rows, all of the target's weight rejected: the draw is from the target after all
    u[0, 1:] = 1.0
    got = check_verify(p, None, np.array([[0, 4999, 4999, 4999]], np.int32), u, star)
    assert got[0][0] == 1 and got[2][0] == 4999
    # no weight anywhere
    got = check_verify(torch.zeros(1, T, V), p, tok, u, star)
    assert got[2][0] == -1
    # out-of-range tokens are rejected and take nothing out
    w = torch.full((1, T, V), 1.0 / V)
    for bad in (-1, V, 2 ** 31 - 1, -2 ** 31):
        check_verify(w, None, np.array([[0, bad, bad, 3]], np.int32), np.array([[0.3, 0.0, 0.0, 0.9]], np.float32), star)
        check_verify(w, w * 2, np.array([[0, bad, bad, 3]], np.int32), np.array([[0.3, 0.0, 0.0, 0.9]], np.float32), star)
    # what is no probability counts as 0, in both
    x = w.clone()
    x[0, :, 10:20] = float("nan"); x[0, :, 20:30] = float("inf"); x[0, :, 30:40] = -1.0
    x[0, :, 40:50] = float("-inf")
    for u0 in (0.0, 0.0021, 0.4):
        for t in (15, 25, 35, 45, 60):
            u = np.array([[u0, 0.5, 0.5, 0.5]], np.float32)
            check_verify(x, w, np.array([[0, t, t, t]], np.int32), u, star)
            check_verify(w, x, np.array([[0, t, t, t]], np.int32), u, star)
            check_verify(x, None, np.array([[0, t, t, t]], np.int32), u, star)


def test_verify_of_a_chain_given_as_a_tree():
    """parents that spell chains out give what no parents give (other kernels)."""
    rng = np.random.default_rng(3)
    N, T, V = 9, 6, 3003
    target, draft = probabilities(rng, N, T, V, BF16)
    tokens = rng.integers(0, V, (N, T)).astype(np.int32)
    tokens[:, 1:] = draft[:, :-1].float().argmax(-1).numpy()
    u = rng.random((N, T)).astype(np.float32)
    for d in (draft, None):
        a = check_verify(target, d, tokens, u, None)
        b = check_verify(target, d, tokens, u, random_parents(N, T, "chain", 0))
        assert [x.tolist() for x in a] == [x.tolist() for x in b]


def test_verify_in_a_workspace_of_a_larger_batch():
    """A batch that shrinks keeps its workspace (the rows are spread over the GPU
    at these sizes, so the workspace holds partial sums)."""
    rng = np.random.default_rng(12)
    T, V = 2, 65536
    ws = kda.verify_workspace(64, 4, V, DEV)
    for N in (63, 17, 1):
        target, draft = probabilities(rng, N, T, V, BF16)
        tokens = draft[:, :1].float().argmax(-1).expand(N, T).numpy().astype(np.int32)
        check_verify(target, draft, tokens, rng.random((N, T)).astype(np.float32), None, workspace=ws)


def test_verify_of_arrays_side_by_side():
    """Inputs and outputs that touch without overlapping, in one buffer."""
    rng = np.random.default_rng(13)
    N, T, V = 5, 7, 900
    target, draft = probabilities(rng, N, T, V, F32)
    tokens, u = rng.integers(0, V, (N, T)).astype(np.int32), rng.random((N, T)).astype(np.float32)
    par, nodes = random_parents(N, T, "bushy", 1), np.full(N, T, np.int32)
    buf = torch.full((3 * N + 3 * N * T,), 7, device=DEV, dtype=torch.int32)
    at = 0
    parts = []
    for shape in ((N,), (N, T), (N, T), (N,), (N, T), (N,)):
        size = int(np.prod(shape))
        parts.append(buf[at:at + size].view(shape))
        at += size
    accept, tok, path, next_token, p, nn = parts
    tok.copy_(dev(tokens, torch.int32)); p.copy_(dev(par, torch.int32)); nn.copy_(dev(nodes, torch.int32))
    got = kda.verify_drafts(target.to(DEV), draft.to(DEV), tok, dev(u), p, nn, accept=accept, path=path, next_token=next_token)
    want = speculative.verify(target.numpy(), draft.numpy(), tokens, u, par, nodes)
    assert all(a.tolist() == b.tolist() for a, b in zip(got, want))
    assert torch.equal(tok, dev(tokens, torch.int32)) and torch.equal(p, dev(par, torch.int32))
    with pytest.raises(kda.KdaError):
        kda.verify_drafts(target.to(DEV), draft.to(DEV), tok, dev(u), p, nn, accept=accept, path=tok, next_token=next_token)


@pytest.mark.parametrize("N,V,tree", [(3, 700, "chain"), (3, 700, "star"), (2, 66001, "chain"), (2, 66001, "star")])
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_of_uniforms_that_are_nan(N, V, tree, with_draft):
    """The kernel reads the NaN itself: a test of NaN accepts nothing, and a draw
    of NaN is one of 0 (the first token of the residual, one of many here)."""
    rng = np.random.default_rng(V)
    T = 4
    target, draft = probabilities(rng, N, T, V, F32)
    target[:, :, :3] = 0.0                                    # the draw of 0 is token 3 or the next one left
    par = random_parents(N, T, tree, 0)
    tokens = rng.integers(4, V, (N, T)).astype(np.int32)
    u = rng.random((N, T)).astype(np.float32) * 0.5
    u[:, 0], u[0, 1:], u[1, 2] = np.nan, np.nan, np.nan
    stand_in = np.where(np.isnan(u), np.float32(1e30), u)     # rejects: every token has weight in both rows
    stand_in[:, 0] = 0.0
    d = draft if with_draft else None
    got = kda.verify_drafts(target.to(DEV), None if d is None else d.to(DEV), dev(tokens, torch.int32), dev(u),
                            None if tree == "chain" else dev(par, torch.int32))
    want = speculative.verify(target.numpy(), None if d is None else d.numpy(), tokens, stand_in, par)
    for a, b in zip(got, want):
        assert a.tolist() == b.tolist()
    assert got[0][0] == 1 and (got[2] >= 3).all() and (got[2] < 3 + 64).all()


def test_verify_rejects_a_near_certain_token_exactly():
    """One token holds all but 2^-60 of a row: without it the residual is the
    rest, which no subtraction of sums may lose."""
    V = 4096
    p = torch.full((1, 2, V), 2.0 ** -72)
    p[0, :, 77] = 1.0
    for u0 in (0.0, 0.25, 0.75):
        got = check_verify(p, None, np.array([[0, 77]], np.int32), np.array([[u0, 1.0]], np.float32), None)
        assert got[0][0] == 1 and got[2][0] != 77
        assert abs(int(got[2][0]) - u0 * V) <= 1


def states(N, H, D, seed):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((N, H, D, D)) * 10.0 ** rng.uniform(-5, 4, (N, H, D, 1))).astype(np.float32)


def check_cache(cache, x, slots):
    """Slots hold exactly what the oracle's rounding of x gives."""
    y, code = speculative.quantise(x, cache.format == kda.CACHE_E4M3)
    got_v = cache.values.float().cpu().numpy().reshape(cache.values.shape[0], cache.values.shape[1], -1)
    got_c = cache.scales.cpu().numpy()
    for n, slot in enumerate(slots):
        np.testing.assert_array_equal(got_c[slot], code[n])
        np.testing.assert_array_equal(got_v[slot], y[n])
    return y, code


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("N,H,D", [(1, 1, 128), (5, 3, 128), (1, 1, 16), (7, 2, 16)])
def test_cache_round_trip(N, H, D, fmt):
    x = states(N, H, D, N + D)
    x[0, 0, 0] = 0.0                                          # blocks of zeros
    x[0, 0, 1, :8] = [1e-45, -1e-45, 1e-38, 3e-39, 0, -0.0, 1e-40, 1e-44]
    x[-1, -1, 5, 3] = 3.4e38                                  # near the largest
    x[-1, 0, 7, :4] = np.float32([127, 126.5, 63.5, -0.5]) * 2.0 ** -9
    cache = kda.make_state_cache(N + 4, H, D, DEV, dtype=fmt)
    slots = np.random.default_rng(1).permutation(N + 4)[:N].astype(np.int32)
    kda.state_store(dev(x), cache, dev(slots, torch.int32))
    y, code = check_cache(cache, x, slots)
    others = sorted(set(range(N + 4)) - set(slots.tolist()))
    assert not cache.values.view(torch.uint8)[others].any() and not cache.scales[others].any()
    back = kda.state_load(cache, dev(slots, torch.int32))
    want = speculative.dequantise(y, code).astype(np.float32).reshape(x.shape)
    np.testing.assert_array_equal(back.cpu().numpy(), want)
    # within half a step of each value
    b = np.abs(back.cpu().numpy().astype(np.float64) - x).reshape(N, H, -1, 32)
    top = np.abs(x).reshape(N, H, -1, 32).max(-1, keepdims=True).astype(np.float64)
    half = (2.0 ** (code.astype(np.float64) - 128))[..., None]
    if fmt is torch.int8:
        assert (b <= half).all() and (b <= np.maximum(top / 127, 2.0 ** -127)).all()
    else:
        assert (b <= np.maximum(2.0 ** -4 * np.abs(x.reshape(b.shape)), half * 2.0 ** -9)).all()
    # all slots, without a list
    everything = kda.state_load(cache)
    assert torch.equal(everything[torch.from_numpy(slots).long().to(DEV)], back)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_cache_slots_outside_twice_and_without_a_list(fmt):
    N, H, D = 6, 2, 128
    x = states(N, H, D, 3)
    cache = kda.make_state_cache(4, H, D, DEV, dtype=fmt)
    # 1 is named three times: the last state wins; -1, 4 and INT32_MAX are outside
    slots = np.array([1, -1, 1, 4, 1, 2 ** 31 - 1], np.int32)
    kda.state_store(dev(x), cache, dev(slots, torch.int32))
    check_cache(cache, x[4:5], [1])
    assert not cache.values.view(torch.uint8)[[0, 2, 3]].any()
    back = torch.full((N, H, D, D), 5.0, device=DEV)
    kda.state_load(cache, dev(slots, torch.int32), states=back)
    want = kda.state_load(cache)[1]
    for n, slot in enumerate(slots):
        assert torch.equal(back[n], want if slot == 1 else torch.zeros_like(want))
    kda.state_store(dev(x[:3]), cache)
    check_cache(cache, x[:3], [0, 1, 2])


@pytest.mark.parametrize("N,H,D,num_slots", [
    (600, 1, 16, 7), (5000, 1, 16, 700), (5000, 2, 16, 6000), (2300, 1, 128, 40), (513, 1, 16, 512), (2049, 1, 128, 1)])
def test_cache_of_long_lists_that_name_slots_again(N, H, D, num_slots):
    x = torch.randn(N, H, D, D, device=DEV, generator=torch.Generator(DEV).manual_seed(N))
    slots = np.random.default_rng(num_slots).integers(0, num_slots, N).astype(np.int32)
    slots[0] = slots[-1]                                      # the first and the last state
    cache, want = (kda.make_state_cache(num_slots, H, D, DEV) for _ in range(2))
    kda.state_store(x, cache, dev(slots, torch.int32))
    last = {int(s): n for n, s in enumerate(slots)}           # each slot's latest state, stored without repeats
    kda.state_store(x[torch.tensor(list(last.values()), device=DEV)], want, dev(np.array(list(last), np.int32), torch.int32))
    assert torch.equal(cache.values, want.values) and torch.equal(cache.scales, want.scales)


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_cache_of_values_that_are_not_finite(fmt):
    x = states(1, 1, 16, 8)
    x[0, 0, 0, :3] = [np.inf, -np.inf, np.nan]                # other values of the block keep their step
    x[0, 0, 4:6] = np.nan
    x[0, 0, 8:10] = np.inf
    cache = kda.make_state_cache(1, 1, 16, DEV, dtype=fmt)
    kda.state_store(dev(x), cache)
    check_cache(cache, x, [0])


def test_cache_reads_every_code():
    """All 256 codes under steps from 2^-127 to 2^128, through the load."""
    for fmt in (torch.int8, torch.float8_e4m3fn):
        cache = kda.make_state_cache(1, 8, 16, DEV, dtype=fmt)
        cache.values.view(torch.uint8).copy_(torch.arange(256, dtype=torch.uint8).reshape(16, 16).expand(1, 8, 16, 16))
        codes = torch.tensor([0, 1, 2, 100, 127, 200, 240, 255], dtype=torch.uint8)
        cache.scales.copy_(codes[None, :, None].expand(1, 8, 8))
        got = kda.state_load(cache).cpu().numpy()
        vals = cache.values.cpu().float().numpy().reshape(1, 8, -1)
        with np.errstate(over="ignore", invalid="ignore"):
            want = speculative.dequantise(vals, cache.scales.cpu().numpy()).astype(np.float32).reshape(got.shape)
        np.testing.assert_array_equal(got, want)


def test_offsets_past_32_bits():
    """States of 4.4 G values, a cache of 2.2 G and rows of 2.2 G probabilities:
    the last sequence gives what it gives alone."""
    N, T, H, D = 4200, 2, 64, 128
    gen = torch.Generator(device=DEV).manual_seed(5)
    one = Step(1, T, H, D, BF16, 6)
    args = [x.expand(N, *x.shape[1:]).contiguous() for x in one.args]
    state = torch.zeros(N, H, D, D, device=DEV)
    state[-1] = one.state[0]
    assert state.numel() > 2 ** 32
    o = kda.decode_tree(*args, state)
    assert torch.equal(o[-1], kda.decode_tree(*one.args, one.state)[0])
    assert torch.equal(o[7], kda.decode_tree(*one.args, torch.zeros_like(one.state))[0])
    path = torch.zeros(N, T, device=DEV, dtype=torch.int32)
    path[:, 1] = 1
    accept = torch.zeros(N, device=DEV, dtype=torch.int32)
    accept[-1] = 2
    kda.commit_path(*args[1:], state, path, accept)
    kda.commit_path(*one.args[1:], one.state, path[-1:], torch.full((1,), 2, device=DEV, dtype=torch.int32))
    assert torch.equal(state[-1], one.state[0])
    cache = kda.make_state_cache(2100, H, D, DEV)
    assert cache.values.numel() > 2 ** 31
    slots = torch.full((1,), 2099, device=DEV, dtype=torch.int32)
    kda.state_store(one.state, cache, slots)
    small = kda.make_state_cache(1, H, D, DEV)
    kda.state_store(one.state, small)
    assert torch.equal(kda.state_load(cache, slots), kda.state_load(small))
    del state, args, o, cache
    N, T, V = 17, 64, 2000003
    target = torch.zeros(N, T, V, device=DEV, dtype=BF16)
    assert target.numel() > 2 ** 31
    target[-1, :, -9:] = torch.rand(T, 9, device=DEV, generator=gen).to(BF16)
    tokens = torch.full((N, T), V - 1, device=DEV, dtype=torch.int32)
    u = torch.rand(N, T, device=DEV, generator=gen)
    u[-1, 1:60] = 0.0
    many = kda.verify_drafts(target, None, tokens, u)
    alone = kda.verify_drafts(target[-1:].contiguous(), None, tokens[-1:], u[-1:].contiguous())
    assert [x[-1].tolist() for x in many] == [x[0].tolist() for x in alone]
    assert int(many[0][-1]) >= 60 and V - 9 <= int(many[2][-1]) < V and many[2][0] == -1


def full_step(s, par, target, draft, tokens, u, nodes, cache, slots, ws):
    """Cached states in, tree, verification, commit, cached states out."""
    state = kda.state_load(cache, slots)
    o = kda.decode_tree(*s.args, state, par, nodes)
    accept, path, token = kda.verify_drafts(target, draft, tokens, u, par, nodes, workspace=ws)
    kda.commit_path(*s.args[1:], state, path, accept)
    kda.state_store(state, cache, slots)
    return o, accept, path, token, state


def step_setup(N=5, T=12, H=2, D=128, V=3001):
    rng = np.random.default_rng(77)
    s = Step(N, T, H, D, BF16, 77)
    par = random_parents(N, T, "bushy", 4)
    target, draft = probabilities(rng, N, T, V, F32)
    tokens = np.zeros((N, T), np.int32)
    for n in range(N):
        for i in range(1, T):
            w = draft[n, par[n, i]].double().numpy()
            tokens[n, i] = rng.choice(V, p=w / w.sum())
    u = rng.random((N, T)).astype(np.float32)
    nodes = np.array([T, T, 0, T - 5, T], np.int32)[:N]
    cache = kda.make_state_cache(N + 2, H, D, DEV)
    slots = dev(np.arange(N)[::-1].astype(np.int32), torch.int32)
    kda.state_store(s.state, cache, slots)
    return (s, dev(par, torch.int32), target.to(DEV), draft.to(DEV), dev(tokens, torch.int32), dev(u),
            dev(nodes, torch.int32), cache, slots, kda.verify_workspace(N, T, V, DEV)), par, tokens, u, nodes


def test_a_step_from_cache_to_cache():
    a, par, tokens, u, nodes = step_setup()
    s, target, draft, cache, slots = a[0], a[2], a[3], a[7], a[8]
    s.s0 = kda.state_load(cache, slots).cpu().numpy()
    o, accept, path, token, state = full_step(*a)
    s.check_tree(o, par, nodes)
    acc, pth, nxt = speculative.verify(target.cpu().numpy(), draft.cpu().numpy(), tokens, u, par, nodes)
    assert accept.tolist() == acc.tolist() and path.tolist() == pth.tolist() and token.tolist() == nxt.tolist()
    ref, size, lengths = speculative.commit_path(s.k, s.v, s.g, s.b, s.s0, pth, acc)
    assert lengths.tolist() == acc.tolist() and lengths.max() > 1
    err = np.sqrt(((host(state) - ref) ** 2).sum(-2))
    assert (err <= lengths[:, None, None] * 144 * 2.0 ** -24 * size).all()
    # the outputs are those of the accepted path run as tokens on the committed prefix
    n = int(np.argmax(acc))
    idx = torch.from_numpy(pth[n, :acc[n]]).long().to(DEV)
    st = dev(s.s0[n:n + 1])
    chain = kda.decode_tokens(*(x[n:n + 1, idx].contiguous() for x in s.args), st)
    s.check_tree(o, par, nodes)
    assert (chain[0].float() - o[n, idx].float()).abs().max() <= 2.0 ** -6 * o[n, idx].float().abs().max()
    # committing the accepted path and decoding its tokens one after the other are the same recurrence
    assert (st[0] - state[n]).norm() <= 2 * acc[n] * 144 * 2.0 ** -24 * float(np.linalg.norm(size[n]))
    check_cache(cache, state.cpu().numpy(), slots.tolist())


def test_a_step_captured_and_replayed():
    """The whole step in one graph, replayed over refreshed inputs with eager
    work between the replays; each replay equals the eager step."""
    a, par, tokens, u, nodes = step_setup()
    s, us, cache = a[0], a[5], a[7]
    first = [cache.values.clone(), cache.scales.clone()]

    def reset():
        cache.values.copy_(first[0])
        cache.scales.copy_(first[1])

    full_step(*a)                                             # loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = full_step(*a)
    for turn in range(4):
        us.copy_(torch.rand(us.shape, generator=torch.Generator().manual_seed(turn)))
        reset()
        want = [x.clone() for x in full_step(*a)]
        kept = [cache.values.clone(), cache.scales.clone()]
        reset()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)
        assert torch.equal(cache.values, kept[0]) and torch.equal(cache.scales, kept[1])


def test_on_another_stream_and_twice_the_same():
    a, *_ = step_setup()
    cache = a[7]
    first = [cache.values.clone(), cache.scales.clone()]
    want = [x.clone() for x in full_step(*a)]
    for _ in range(3):
        cache.values.copy_(first[0]); cache.scales.copy_(first[1])
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            got = full_step(*a)
        torch.cuda.current_stream().wait_stream(stream)
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_two_steps_at_once():
    """Two steps with their own caches and workspaces on two streams, over and
    over: each gives what it gives alone."""
    steps, wants, firsts = [step_setup()[0], step_setup(N=4, T=9)[0]], [], []
    for a in steps:
        cache = a[7]
        firsts.append([cache.values.clone(), cache.scales.clone()])
        wants.append([x.clone() for x in full_step(*a)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for a, first, stream in zip(steps, firsts, streams):
            with torch.cuda.stream(stream):
                a[7].values.copy_(first[0])
                a[7].scales.copy_(first[1])
                got.append(full_step(*a))
        torch.cuda.synchronize()
        for want, out in zip(wants, got):
            for x, y in zip(want, out):
                assert torch.equal(x, y)


def test_empty_calls():
    x = torch.empty(0, 4, 2, 128, device=DEV, dtype=BF16)
    g, b, st = torch.empty(0, 4, 2, 128, device=DEV), torch.empty(0, 4, 2, device=DEV), torch.empty(0, 2, 128, 128, device=DEV)
    assert kda.decode_tree(x, x, x, g, b, st).shape == x.shape
    i = torch.empty(0, 4, device=DEV, dtype=torch.int32)
    kda.commit_path(x, x, g, b, st, i, torch.empty(0, device=DEV, dtype=torch.int32))
    p = torch.empty(0, 4, 100, device=DEV)
    assert kda.verify_drafts(p, p, i, torch.empty(0, 4, device=DEV))[1].shape == (0, 4)
    cache = kda.make_state_cache(2, 2, 128, DEV)
    kda.state_store(st, cache, torch.empty(0, device=DEV, dtype=torch.int32))
    assert kda.state_load(cache, torch.empty(0, device=DEV, dtype=torch.int32)).shape == (0, 2, 128, 128)
