"""The training calls together, as examples/train_step.py runs them: the
gradients of a whole fp32 layer against central differences of the same
layer's formulas in 64 bits, and against the formulas themselves; a bf16 layer
against the formulas; and a short training run."""
import os
import sys

import numpy as np
import pytest
import torch

import train_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def _host(t):
    return t.detach().double().cpu().numpy()


def _rel(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


def _run(cfg, T, capacity):
    from train_step import TrainLayer
    L = TrainLayer(cfg, T, capacity=capacity, balance=0.1, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(T, cfg.d, device="cuda", generator=gen).to(L.out.dtype)
    r = torch.randn(T, cfg.d, device="cuda", generator=gen).to(L.out.dtype)
    L.forward(x)
    L.backward(x, r)
    L.check()
    return L, x, r


def _formulas(L, x, r):
    """The layer's loss as a function of x and its weights, with the routing
    decision (expert indices, dropped slots) held as the layer took it, and
    the gradients by the formulas; all in 64 bits."""
    cfg, k, T = L.cfg, L.cfg.k, L.T
    idx = L.topk_idx.cpu().numpy()
    off, perm, inv = ref.sort_slots(idx, cfg.N, L.capacity)
    kept_idx = np.where(inv >= 0, idx, -1)
    # the gates are renormalised over the token's choices, dropped ones included
    load = ref.load_of(idx, cfg.N)
    r = _host(r)

    def forward(x, wr, wg, wu, wd, full=False):
        l = x @ wr.T
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        gate = ref.gates(p, idx, True)
        xp = ref.dispatch(x, perm, k)
        g, u, h, _, _ = ref.experts_up(xp, off, wg, wu)
        y, _ = ref.experts_down(h, off, wd)
        out, _ = ref.combine(y, gate, inv, None)
        loss = float((r * out).sum()) + ref.balance_loss(p, load, L.balance)
        return (loss, p, gate, xp, g, u, h, y, out) if full else loss

    at = [_host(t) for t in (x, L.w_router, L.w_gate, L.w_up, L.w_down)]
    _, p, gate, xp, g, u, h, y, out = forward(*at, full=True)
    dy, dgate, _ = ref.combine_grad(r, y, gate, inv)
    dg, du, _, _ = ref.experts_dh(dy, g, u, off, at[4])
    dxp, _ = ref.experts_dx(dg, du, off, at[2], at[3])
    dl, _, _ = ref.gate_grad(p, idx, np.where(kept_idx >= 0, dgate, 0.0), True, L.balance)
    dx = ref.combine(dxp, None, inv, None)[0] + dl @ at[1]
    grads = [dx, dl.T @ at[0], ref.experts_dw(dg, xp, off, cfg.N)[0], ref.experts_dw(du, xp, off, cfg.N)[0],
             ref.experts_dw(h, dy, off, cfg.N)[0]]
    return forward, at, grads, out


# float32 sums of up to 512 terms (and the router's float32 logits) leave relative
# errors of some 1e-6 in every stage; the chain has four.  bf16 rounds at ten places
# on the longest path, each by up to 2^-8 and 2^-8 / sqrt(3) on average.
TOL = {"f32": 2e-5, "bf16": 1e-2 * np.sqrt(10.0)}


@pytest.mark.parametrize("layer,T,capacity", [("tiny", 16, 0), ("tiny", 33, 5), ("granite", 48, 0), ("granite", 130, 30)])
def test_gradients_of_a_whole_layer(layer, T, capacity):
    from workloads import CONFIGS
    L, x, r = _run(CONFIGS[layer], T, capacity)
    forward, at, grads, out = _formulas(L, x, r)
    tol = TOL[L.cfg.wtype]
    got = [L.dx, L.dw_router, L.dw_gate, L.dw_up, L.dw_down]
    assert _rel(_host(L.out), out) <= tol
    for name, a, b in zip(("dx", "dw_router", "dw_gate", "dw_up", "dw_down"), got, grads):
        assert _rel(_host(a), b) <= tol, name
    if L.cfg.wtype == "f32":  # differences along random directions; truncation (1e-4)^2, cancellation 1e-16 / 1e-4
        rng = np.random.default_rng(0)
        for i, a in enumerate(got):
            v = rng.standard_normal(at[i].shape) * (1.0 if i == 0 else 0.02)
            f = lambda s: forward(*[z + s * v if j == i else z for j, z in enumerate(at)])  # noqa: E731
            slope = (f(1e-4) - f(-1e-4)) / 2e-4
            # the gradient's error is at most tol of its norm, so its product with v is off by no more than
            assert abs(float((_host(a) * v).sum()) - slope) <= tol * np.linalg.norm(grads[i]) * np.linalg.norm(v) + 1e-6


def test_accumulation_over_two_micro_batches():
    from workloads import CONFIGS
    L, x, r = _run(CONFIGS["tiny"], 16, 0)
    once = [t.clone() for t in (L.dw_router, L.dw_gate, L.dw_up, L.dw_down)]
    L.backward(x, r, accumulate=True)
    for a, b in zip((L.dw_router, L.dw_gate, L.dw_up, L.dw_down), once):
        assert _rel(_host(a), 2 * _host(b)) <= 1e-6


@pytest.mark.parametrize("layer,tokens", [("tiny", 64), ("granite", 200)])
def test_training_lowers_the_loss(layer, tokens):
    from train_step import train
    losses = train(layer, tokens, steps=12)
    assert all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
