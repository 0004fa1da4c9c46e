"""The training step's kernels against the plain 64-bit implementations of
train_ref, within its derived bounds (sorted indices and zero rows exactly)."""
import numpy as np
import pytest
import torch

import expert_routing_ffn_gb300 as moe
import train_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def rnd(rng, shape, kind, sd=1.0):
    """Values of the type: (device tensor, exact float64 copy)"""
    t = torch.from_numpy((rng.standard_normal(shape) * sd).astype(np.float32)).to(TYPES[kind])
    return t.cuda(), t.double().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def ints(t):
    return t.cpu().numpy()


def empty(shape, kind):
    """An output buffer of NaN: every value has to be written."""
    return torch.full(shape, float("nan"), dtype=TYPES[kind], device="cuda")


def workspace(D):
    return torch.zeros(moe.moe_train_workspace_size(D), dtype=torch.uint8, device="cuda")


def routing(rng, T, N, k, how):
    """expert_idx [T, k]: distinct experts a token, `how` says which slots have none."""
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    if how == "one":      # every first choice on one expert
        for t in range(T):
            at = np.nonzero(idx[t] == N // 2)[0]
            idx[t, at[0] if at.size else 0] = idx[t, 0]
            idx[t, 0] = N // 2
    elif how == "none":
        idx[:] = -1
    elif how == "some":
        idx[rng.random(idx.shape) < 0.3] = -1
        if T > 2:
            idx[1] = -1   # a token without any expert
    elif how == "skew":
        p = 1.0 / np.arange(1, N + 1) ** 1.1
        idx = np.stack([rng.choice(N, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)
    return idx


def clean(ws):
    st, det = moe.moe_check(ws)
    assert st == moe.MOE_OK, (moe.status_string(st), det)


# ---------------------------------------------------------------- dispatch

ROWS = [  # T, d, N, k, routing, capacity, type
    (1, 2048, 64, 6, "all", 0, "bf16"), (1, 1, 1, 1, "all", 0, "bf16"), (1, 7, 3, 1, "none", 0, "f32"),
    (2, 64, 8, 2, "all", 1, "bf16"), (33, 250, 40, 8, "some", 0, "bf16"), (33, 251, 40, 8, "some", 3, "bf16"),
    (257, 1000, 40, 8, "skew", 60, "f32"), (300, 96, 65, 3, "one", 100, "bf16"), (64, 40, 300, 16, "all", 0, "f32"),
    (700, 33, 512, 16, "skew", 20, "f32"), (1025, 64, 64, 1, "one", 0, "bf16"), (2500, 24, 60, 7, "some", 250, "bf16"),
    (9000, 8, 16, 8, "skew", 3000, "f32"), (70000, 2, 5, 1, "some", 0, "bf16"), (129, 3584, 64, 8, "all", 0, "bf16"),
]


@pytest.mark.parametrize("T,d,N,k,how,cap,kind", ROWS)
def test_dispatch_sorts_and_copies(T, d, N, k, how, cap, kind):
    rng = np.random.default_rng(T * 31 + d)
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    x, xh = rnd(rng, (T, d), kind)
    idx = routing(rng, T, N, k, how)
    ws = workspace(D)
    xp = empty((T * k, d), kind)
    off, perm, inv = (torch.full((n,), -77, dtype=torch.int32, device="cuda") for n in (N + 1, T * k, T * k))
    moe.moe_dispatch_rows(D, x, dev(idx), cap, xp, off, perm, inv, ws)
    clean(ws)
    roff, rperm, rinv = ref.sort_slots(idx, N, cap)
    assert np.array_equal(ints(off), roff)
    assert np.array_equal(ints(perm), rperm)
    assert np.array_equal(ints(inv).reshape(T, k), rinv)
    assert np.array_equal(host(xp), ref.dispatch(xh, rperm, k))


def test_dispatch_reports_an_expert_out_of_range_and_goes_on():
    D = moe.make_dims(3, 16, 4, 2, 64, wtype="f32")
    rng = np.random.default_rng(5)
    x, xh = rnd(rng, (3, 16), "f32")
    idx = np.array([[0, 4], [3, 1], [1 << 30, 2]], np.int32)
    ws = workspace(D)
    xp, off, perm, inv = empty((6, 16), "f32"), *(torch.zeros(n, dtype=torch.int32, device="cuda") for n in (5, 6, 6))
    moe.moe_dispatch_rows(D, x, dev(idx), 0, xp, off, perm, inv, ws)
    st, det = moe.moe_check(ws)
    assert st == moe.MOE_ERR_DEVICE_INDEX and det in (1, 4)
    roff, rperm, rinv = ref.sort_slots(np.where(idx < 4, idx, -1), 4, 0)
    assert np.array_equal(ints(off), roff) and np.array_equal(ints(perm), rperm)
    assert np.array_equal(host(xp), ref.dispatch(xh, rperm, 2))


def test_empty_batch():
    D = moe.make_dims(0, 16, 4, 2, 8, wtype="f32")
    ws = workspace(D)
    z, i0 = torch.zeros((0, 16), device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    off = torch.full((5,), 9, dtype=torch.int32, device="cuda")
    moe.moe_dispatch_rows(D, z, i0, 0, z, off, i0, i0, ws)
    assert ints(off).tolist() == [0] * 5
    moe.moe_combine_rows(D, z, None, i0, None, z)
    moe.moe_dispatch_rows_grad(D, z, i0, None, z)
    loss = torch.ones(1, device="cuda")
    moe.moe_gate_grad(D, z, i0, z, 0.5, z, loss, ws)
    assert loss.item() == 0.0
    w = torch.ones((4, 8, 16), device="cuda")
    h0 = torch.zeros((0, 8), device="cuda")
    moe.moe_experts_up(D, z, off, w, w, None, None, h0, ws)
    dw, dw2 = torch.full_like(w, float("nan")), torch.full_like(w, float("nan"))
    moe.moe_experts_up_grad(D, h0, h0, z, off, w, w, z, dw, dw2, False, ws)
    assert not dw.any() and not dw2.any()  # an expert without rows: zero gradients
    dw.fill_(3.0)
    moe.moe_experts_down_grad(D, z, h0, h0, h0, off, w, h0, h0, dw, True, ws)
    assert bool((dw == 3.0).all())
    clean(ws)


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("T,d,N,k,how,cap,kind", [r for r in ROWS if r[0] < 5000])
@pytest.mark.parametrize("with_add", [False, True])
def test_combine_and_dispatch_gradient(T, d, N, k, how, cap, kind, with_add):
    rng = np.random.default_rng(T * 7 + d)
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    _, _, inv = ref.sort_slots(routing(rng, T, N, k, how), N, cap)
    y, yh = rnd(rng, (T * k, d), kind)
    add, addh = rnd(rng, (T, d), kind) if with_add else (None, None)
    gate = rng.random((T, k)).astype(np.float32)
    gate[inv < 0] = np.nan  # never looked at
    dinv, out = dev(inv), empty((T, d), kind)
    moe.moe_combine_rows(D, y, dev(gate), dinv, add, out)
    exact, mag = ref.combine(yh, gate.astype(np.float64), inv, addh)
    ref.check(host(out), exact, ref.bound(exact, k + 1, mag, kind), "out")
    if T > 1 and not with_add:
        empty_tokens = (inv < 0).all(1)
        assert not host(out)[empty_tokens].any()
    moe.moe_dispatch_rows_grad(D, y, dinv, add, out)
    exact, mag = ref.combine(yh, None, inv, addh)
    ref.check(host(out), exact, ref.bound(exact, k + 1, mag, kind), "dx")


@pytest.mark.parametrize("T,d,N,k,how,cap,kind", [r for r in ROWS if r[0] < 5000])
def test_combine_gradient(T, d, N, k, how, cap, kind):
    rng = np.random.default_rng(T * 5 + d)
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    _, _, inv = ref.sort_slots(routing(rng, T, N, k, how), N, cap)
    y, yh = rnd(rng, (T * k, d), kind)
    kept = int((inv >= 0).sum())
    y[kept:] = float("nan")  # rows of no expert are not read
    dout, dh = rnd(rng, (T, d), kind)
    gate = rng.random((T, k)).astype(np.float32)
    dy, dgate = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad(D, dout, y, dev(gate), dev(inv), dy, dgate)
    edy, edg, mag = ref.combine_grad(dh, np.where(np.arange(T * k)[:, None] < kept, yh, 0.0), gate.astype(np.float64), inv)
    ref.check(host(dy), edy, ref.bound(edy, 1, np.abs(edy), kind), "dy")
    ref.check(host(dgate), edg, ref.bound(edg, d, mag, "f32"), "dgate")
    # each output alone
    dy2, dgate2 = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad(D, dout, None, dev(gate), dev(inv), dy2, None)
    moe.moe_combine_rows_grad(D, dout, y, None, dev(inv), None, dgate2)
    assert torch.equal(dy2, dy) and torch.equal(dgate2, dgate)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("d,ld,shift", [(48, 64, 0), (48, 51, 0), (40, 48, 1), (33, 40, 2)])
def test_token_rows_with_strides_and_odd_starts(kind, d, ld, shift):
    """x, add, out, dx and dout as columns of wider tensors, at any element
    offset; in-place accumulation onto add."""
    T, N, k = 37, 8, 3
    rng = np.random.default_rng(d + ld)
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    idx = routing(rng, T, N, k, "some")
    off, perm, inv = ref.sort_slots(idx, N, 0)

    def wide(t):
        w = torch.full((T, ld + 4), 7.0, dtype=TYPES[kind], device="cuda")
        w[:, shift:shift + d] = t
        return w, w[:, shift:shift + d]

    x, xh = rnd(rng, (T, d), kind)
    _, xv = wide(x)
    ws, xp = workspace(D), empty((T * k, d), kind)
    doff, dperm, dinv = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (N + 1, T * k, T * k))
    moe.moe_dispatch_rows(D, xv, dev(idx), 0, xp, doff, dperm, dinv, ws)
    assert np.array_equal(host(xp), ref.dispatch(xh, perm, k))
    gate = rng.random((T, k)).astype(np.float32)
    frame, acc = wide(x)
    moe.moe_combine_rows(D, xp, dev(gate), dinv, acc, acc)
    exact, mag = ref.combine(ref.dispatch(xh, perm, k), gate.astype(np.float64), inv, xh)
    ref.check(host(acc), exact, ref.bound(exact, k + 1, mag, kind), "out onto add")
    frame[:, shift:shift + d] = 7.0
    assert bool((frame == 7.0).all())  # nothing outside the columns was written
    dy, dgate = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad(D, xv, xp, dev(gate), dinv, dy, dgate)
    edy, edg, mag = ref.combine_grad(xh, ref.dispatch(xh, perm, k), gate.astype(np.float64), inv)
    ref.check(host(dy), edy, ref.bound(edy, 1, np.abs(edy), kind), "dy")
    ref.check(host(dgate), edg, ref.bound(edg, d, mag, "f32"), "dgate")


def test_infinities_and_nan_reach_only_their_own_token():
    T, d, N, k = 6, 32, 4, 2
    rng = np.random.default_rng(3)
    D = moe.make_dims(T, d, N, k, 64, wtype="f32")
    _, _, inv = ref.sort_slots(routing(rng, T, N, k, "all"), N, 0)
    y, yh = rnd(rng, (T * k, d), "f32")
    y[inv[2, 0]] = float("inf")
    y[inv[4, 1]] = float("nan")
    out = empty((T, d), "f32")
    moe.moe_combine_rows(D, y, None, dev(inv), None, out)
    o = host(out)
    assert np.isinf(o[2]).all() and np.isnan(o[4]).all()
    rest = [0, 1, 3, 5]
    exact, mag = ref.combine(yh, None, inv, None)
    ref.check(o[rest], exact[rest], ref.bound(exact, k, mag, "f32")[rest], "the other tokens")


def test_indices_of_the_layers_own_permutation_serve():
    """moe_permute marks a slot without a row by -1: no row is written or read for it."""
    T, d, k = 4, 16, 2
    rng = np.random.default_rng(8)
    D = moe.make_dims(T, d, 4, k, 64, wtype="f32")
    inv = np.array([[0, -1], [1, 2], [-1, -1], [3, 4]], np.int32)
    y, yh = rnd(rng, (T * k, d), "f32")
    dout, dh = rnd(rng, (T, d), "f32")
    out, dy, dgate = empty((T, d), "f32"), empty((T * k, d), "f32"), empty((T, k), "f32")
    moe.moe_combine_rows(D, y, None, dev(inv), None, out)
    exact, mag = ref.combine(yh, None, inv, None)
    ref.check(host(out), exact, ref.bound(exact, k, mag, "f32"), "out")
    moe.moe_combine_rows_grad(D, dout, y, None, dev(inv), dy, dgate)
    edy, edg, mag = ref.combine_grad(dh, yh, None, inv)
    assert np.array_equal(host(dy)[:5], edy[:5]) and np.isnan(host(dy)[5:]).all()
    ref.check(host(dgate), edg, ref.bound(edg, d, mag, "f32"), "dgate")


# ---------------------------------------------------------------- router

@pytest.mark.parametrize("T,N,k,how", [(1, 1, 1, "all"), (1, 64, 6, "all"), (7, 8, 2, "some"), (40, 40, 8, "none"),
                                       (33, 65, 16, "some"), (500, 40, 8, "skew"), (3000, 130, 4, "some"),
                                       (100, 512, 16, "all"), (5000, 7, 3, "one")])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("balance", [0.0, 0.01])
def test_gate_gradient(T, N, k, how, renorm, balance):
    rng = np.random.default_rng(T + N + k)
    D = moe.make_dims(T, 16, N, k, 8, wtype="bf16", renorm_topk=int(renorm))
    logits = rng.standard_normal((T, N)) * 2
    prob = (np.exp(logits) / np.exp(logits).sum(1, keepdims=True)).astype(np.float32)
    if T > 4:
        prob[3] = 0.0   # a row that underflowed: no gates, no gradient
    idx = routing(rng, T, N, k, how)
    dgate = rng.standard_normal((T, k)).astype(np.float32)
    dgate_nan = np.where(idx < 0, np.float32(np.nan), dgate)
    ws, dl, loss = workspace(D), empty((T, N), "f32"), empty((1,), "f32")
    moe.moe_gate_grad(D, dev(prob), dev(idx), dev(dgate_nan), balance, dl, loss, ws)
    clean(ws)
    edl, eloss, mag = ref.gate_grad(prob.astype(np.float64), idx, dgate.astype(np.float64), renorm, balance)
    # the sums over a token's slots and over N experts, and the batch's load terms
    ref.check(host(dl), edl, ref.bound(edl, N + 2 * k + 64, mag, "f32"), "dlogits")
    eloss = np.array([eloss])
    ref.check(host(loss), eloss, ref.bound(eloss, T + N + 64, np.abs(eloss), "f32"), "loss")
    dl2 = empty((T, N), "f32")
    moe.moe_gate_grad(D, dev(prob), dev(idx), dev(dgate_nan), balance, dl2, None, ws)
    assert torch.equal(dl, dl2)


# ---------------------------------------------------------------- experts

FFN = [  # T, d, N, k, I, routing, type
    (1, 256, 8, 2, 64, "all", "bf16"), (1, 8, 1, 1, 8, "all", "bf16"), (3, 40, 5, 2, 24, "some", "bf16"),
    (2, 64, 4, 2, 64, "none", "bf16"), (16, 256, 8, 2, 512, "all", "f32"), (9, 37, 6, 3, 29, "some", "f32"),
    (21, 37, 6, 3, 29, "some", "bf16"), (130, 72, 3, 2, 136, "one", "bf16"), (200, 200, 16, 4, 328, "skew", "bf16"),
    (300, 520, 4, 2, 264, "skew", "bf16"), (65, 1024, 3, 1, 192, "one", "bf16"), (40, 64, 200, 4, 72, "skew", "bf16"),
    (500, 128, 2, 2, 256, "all", "bf16"), (700, 136, 9, 4, 200, "some", "bf16"), (260, 320, 5, 3, 72, "some", "f32"),
    (1100, 384, 2, 1, 320, "one", "bf16"),
]


class Ffn:
    def __init__(self, T, d, N, k, I, how, kind, seed=0):
        rng = self.rng = np.random.default_rng(seed + T * 13 + d + I)
        self.D = moe.make_dims(T, d, N, k, I, wtype=kind)
        self.kind, self.M, self.N, self.d, self.I = kind, T * k, N, d, I
        self.off, _, _ = ref.sort_slots(routing(rng, T, N, k, how), N, 0)
        self.kept = int(self.off[-1])
        self.doff, self.ws = dev(self.off), workspace(self.D)
        self.x, self.xh = self.rows(d)
        (self.wg, self.wgh), (self.wu, self.wuh), (self.wd, self.wdh) = \
            (rnd(rng, (N, I, d), kind, 1.0 / np.sqrt(d)) for _ in range(3))

    def rows(self, n, sd=1.0):
        """Grouped rows; those of no expert hold NaN, which nothing may read."""
        t, h = rnd(self.rng, (self.M, n), self.kind, sd)
        t[self.kept:] = float("nan")
        h[self.kept:] = 0.0
        return t, h

    def done(self):
        clean(self.ws)


@pytest.mark.parametrize("case", FFN, ids=lambda c: "-".join(map(str, c)))
def test_experts_up(case):
    f = Ffn(*case)
    g, u, h, h2 = (empty((f.M, f.I), f.kind) for _ in range(4))
    moe.moe_experts_up(f.D, f.x, f.doff, f.wg, f.wu, g, u, h, f.ws)
    moe.moe_experts_up(f.D, f.x, f.doff, f.wg, f.wu, None, None, h2, f.ws)
    f.done()
    eg, eu, eh, mg, mu = ref.experts_up(f.xh, f.off, f.wgh, f.wuh)
    ref.check(host(g), eg, ref.bound(eg, f.d, mg, f.kind), "g")
    ref.check(host(u), eu, ref.bound(eu, f.d, mu, f.kind), "u")
    ref.check(host(h), eh, ref.up_h_limit(eg, eu, eh, mg, mu, f.d, f.kind), "h")
    assert torch.equal(h, h2)


@pytest.mark.parametrize("case", FFN, ids=lambda c: "-".join(map(str, c)))
def test_experts_down(case):
    f = Ffn(*case)
    h, hh = f.rows(f.I)
    y = empty((f.M, f.d), f.kind)
    moe.moe_experts_down(f.D, h, f.doff, f.wd, y, f.ws)
    f.done()
    ey, mag = ref.experts_down(hh, f.off, f.wdh)
    ref.check(host(y), ey, ref.bound(ey, f.I, mag, f.kind), "y")


@pytest.mark.parametrize("case", FFN, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("gkind", ["own", "f32"])
def test_experts_up_gradient(case, gkind):
    f = Ffn(*case)
    gkind = f.kind if gkind == "own" else "f32"
    (dg, dgh), (du, duh) = f.rows(f.I), f.rows(f.I)
    dx, dwg, dwu = empty((f.M, f.d), f.kind), empty((f.N, f.I, f.d), gkind), empty((f.N, f.I, f.d), gkind)
    moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, f.wg, f.wu, dx, dwg, dwu, False, f.ws)
    f.done()
    edx, mag = ref.experts_dx(dgh, duh, f.off, f.wgh, f.wuh)
    ref.check(host(dx), edx, ref.bound(edx, 2 * f.I, mag, f.kind), "dx")
    for name, got, a in (("dw_gate", dwg, dgh), ("dw_up", dwu, duh)):
        e, mag, n = ref.experts_dw(a, f.xh, f.off, f.N)
        ref.check(host(got), e, ref.bound(e, n, mag, gkind), name)
        none = np.diff(f.off) == 0
        assert not host(got)[none].any()
    # each output alone gives the same bits
    dx2, dwg2, dwu2 = torch.empty_like(dx), torch.empty_like(dwg), torch.empty_like(dwu)
    moe.moe_experts_up_grad(f.D, dg, du, None, f.doff, f.wg, f.wu, dx2, None, None, False, f.ws)
    moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, None, None, None, dwg2, dwu2, False, f.ws)
    assert torch.equal(dx, dx2) and torch.equal(dwg, dwg2) and torch.equal(dwu, dwu2)


@pytest.mark.parametrize("case", FFN, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("gkind", ["own", "f32"])
def test_experts_down_gradient(case, gkind):
    f = Ffn(*case)
    gkind = f.kind if gkind == "own" else "f32"
    (dy, dyh), (h, hh), (g, gh), (u, uh) = f.rows(f.d), f.rows(f.I), f.rows(f.I, 2.0), f.rows(f.I)
    if f.kept > 3:  # far into both tails of the sigmoid
        g[0], gh[0] = 96.0, 96.0
        g[1], gh[1] = -96.0, -96.0
    dg, du, dwd = empty((f.M, f.I), f.kind), empty((f.M, f.I), f.kind), empty((f.N, f.I, f.d), gkind)
    moe.moe_experts_down_grad(f.D, dy, h, g, u, f.doff, f.wd, dg, du, dwd, False, f.ws)
    f.done()
    edg, edu, og, ou = ref.experts_dh(dyh, gh, uh, f.off, f.wdh)
    ref.check(host(dg), edg, ref.rounded(edg, og, f.kind), "dg")
    ref.check(host(du), edu, ref.rounded(edu, ou, f.kind), "du")
    e, mag, n = ref.experts_dw(hh, dyh, f.off, f.N)
    ref.check(host(dwd), e, ref.bound(e, n, mag, gkind), "dw_down")


@pytest.mark.parametrize("case", [c for c in FFN if c[0] in (3, 9, 200, 700)], ids=lambda c: "-".join(map(str, c)))
def test_weight_gradients_accumulate_in_float32(case):
    f = Ffn(*case)
    (dg, dgh), (du, duh), (dy, dyh) = f.rows(f.I), f.rows(f.I), f.rows(f.d)
    olds = [rnd(f.rng, (f.N, f.I, f.d), "f32") for _ in range(3)]
    new = [t.clone() for t, _ in olds]
    moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, f.wg, f.wu, None, new[0], new[1], True, f.ws)
    moe.moe_experts_down_grad(f.D, dy, dg, None, None, f.doff, f.wd, None, None, new[2], True, f.ws)
    f.done()
    for got, (_, old), (a, b) in zip(new, olds, ((dgh, f.xh), (duh, f.xh), (dgh, dyh))):
        e, mag, n = ref.experts_dw(a, b, f.off, f.N)
        ref.check(host(got), e + old, ref.bound(e + old, n + 1, mag + np.abs(old), "f32"), "accumulated")
        none = np.diff(f.off) == 0
        assert np.array_equal(host(got)[none], old[none])


def test_infinities_and_nan_reach_only_their_own_rows_and_experts():
    """A bad row of one expert leaves every other row of the products, and
    every other expert's weight gradient, as they were."""
    f = Ffn(150, 64, 4, 2, 72, "all", "bf16")
    e = 1
    r0, r1 = int(f.off[e]), int(f.off[e + 1])
    (dg, dgh), (du, duh) = f.rows(f.I), f.rows(f.I)
    f.x[r1 - 1], f.x[r0, ::2] = float("nan"), float("inf")
    dg[r1 - 1], du[r0] = float("nan"), float("-inf")
    g, u, h = (empty((f.M, f.I), f.kind) for _ in range(3))
    moe.moe_experts_up(f.D, f.x, f.doff, f.wg, f.wu, g, u, h, f.ws)
    dx, dwg, dwu = empty((f.M, f.d), f.kind), empty((f.N, f.I, f.d), "f32"), empty((f.N, f.I, f.d), "f32")
    moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, f.wg, f.wu, dx, dwg, dwu, False, f.ws)
    f.done()
    rows = [i for i in range(f.M) if i not in (r0, r1 - 1)]
    assert np.isfinite(host(g)[rows]).all() and np.isfinite(host(h)[rows]).all() and np.isfinite(host(dx)[rows]).all()
    assert np.isnan(host(g)[r1 - 1]).all() and np.isnan(host(dx)[r1 - 1]).all()
    others = [i for i in range(f.N) if i != e]
    assert np.isfinite(host(dwg)[others]).all() and np.isfinite(host(dwu)[others]).all()
    ex, mag, n = ref.experts_dw(dgh, np.where(np.arange(f.M)[:, None] < f.kept, f.xh, 0.0), f.off, f.N)
    ref.check(host(dwg)[others], ex[others], ref.bound(ex, n, mag, "f32")[others], "the other experts' dw_gate")


def test_unaligned_buffers_of_an_aligned_size():
    """Sizes that the tensor cores take at addresses they cannot: same results."""
    f = Ffn(50, 64, 4, 2, 72, "some", "bf16")
    n = f.wg.numel()
    room = torch.zeros(n + 3, dtype=torch.bfloat16, device="cuda")
    w = room[3:3 + n].view_as(f.wg)
    w.copy_(f.wg)
    g, u, h = (empty((f.M, f.I), f.kind) for _ in range(3))
    moe.moe_experts_up(f.D, f.x, f.doff, w, f.wu, g, u, h, f.ws)
    f.done()
    eg, eu, eh, mg, mu = ref.experts_up(f.xh, f.off, f.wgh, f.wuh)
    ref.check(host(g), eg, ref.bound(eg, f.d, mg, f.kind), "g")
    ref.check(host(h), eh, ref.up_h_limit(eg, eu, eh, mg, mu, f.d, f.kind), "h")


def test_calls_on_a_side_stream_and_repeated_calls_agree():
    f = Ffn(300, 520, 4, 2, 264, "skew", "bf16")
    (dg, _), (du, _) = f.rows(f.I), f.rows(f.I)

    def once(stream):
        out = [empty((f.M, f.I), f.kind) for _ in range(3)] + [empty((f.M, f.d), f.kind)] + \
            [empty((f.N, f.I, f.d), "f32") for _ in range(2)]
        torch.cuda.synchronize()
        moe.moe_experts_up(f.D, f.x, f.doff, f.wg, f.wu, *out[:3], f.ws, stream=stream)
        moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, f.wg, f.wu, *out[3:], False, f.ws, stream=stream)
        torch.cuda.synchronize()
        return out

    first = once(None)
    for stream in (torch.cuda.Stream(), None):
        assert all(torch.equal(a, b) for a, b in zip(first, once(stream)))
    f.done()


def test_calls_replay_from_a_graph():
    T, d, N, k, I = 200, 256, 8, 2, 128
    rng = np.random.default_rng(1)
    D = moe.make_dims(T, d, N, k, I, wtype="bf16")
    x, _ = rnd(rng, (T, d), "bf16")
    idx = dev(routing(rng, T, N, k, "some"))
    (wg, _), (wu, _), (wd, _) = (rnd(rng, (N, I, d), "bf16", 0.06) for _ in range(3))
    gate, ws = torch.rand((T, k), device="cuda"), workspace(D)
    xp, y = empty((T * k, d), "bf16"), empty((T * k, d), "bf16")
    g, u, h = (empty((T * k, I), "bf16") for _ in range(3))
    off, perm, inv = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (N + 1, T * k, T * k))
    out = empty((T, d), "bf16")

    def step():
        moe.moe_dispatch_rows(D, x, idx, 0, xp, off, perm, inv, ws)
        moe.moe_experts_up(D, xp, off, wg, wu, g, u, h, ws)
        moe.moe_experts_down(D, h, off, wd, y, ws)
        moe.moe_combine_rows(D, y, gate, inv, None, out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2, _ = rnd(rng, (T, d), "bf16")
    x.copy_(x2)
    idx.copy_(dev(routing(rng, T, N, k, "all")))
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(out, replayed)
    clean(ws)
