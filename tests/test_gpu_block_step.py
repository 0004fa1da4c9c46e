"""The block and the packed activations together, as examples/train_step.py
runs them: a whole block's gradients against the formulas in 64 bits on what
the step keeps, the same step in a graph, and the block's end behind the
inference layer."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
import train_ref as tr
from test_gpu_packed import values
from test_gpu_train_step import TOL, _host, _rel
from workloads import CONFIGS

pytestmark = pytest.mark.gpu


def _run(layer, T, packed, capacity=0):
    from train_step import TrainBlock
    L = TrainBlock(CONFIGS[layer], T, capacity=capacity, balance=0.1, seed=3, packed=packed)
    gen = torch.Generator("cuda").manual_seed(4)
    x, r1, r2 = (torch.randn(T, L.cfg.d, device="cuda", generator=gen).to(L.out.dtype) for _ in range(3))
    for w in (L.w_pre, L.w_post, L.w_next, L.w_chan):
        w += 0.2 * torch.randn(L.cfg.d, device="cuda", generator=gen).to(w.dtype)
    L.forward(x)
    L.backward(x, r2, dstream=r1)
    L.check()
    return L, x, r1, r2


@pytest.mark.parametrize("layer,T,capacity", [("tiny", 16, 0), ("tiny", 33, 5), ("granite", 48, 0), ("granite", 130, 30)])
@pytest.mark.parametrize("packed", [False, True])
def test_gradients_of_a_whole_block(layer, T, capacity, packed):
    L, x, r1, r2 = _run(layer, T, packed, capacity)
    cfg, k, tol = L.cfg, L.cfg.k, TOL[L.cfg.wtype]
    eps, scale = float(np.float32(1e-6)), 0.5
    x, r1, r2 = _host(x), _host(r1), _host(r2)
    wr, wg, wu, wd, wpre, wpost, wnext, wchan = (_host(w) for w, _ in L.weights())
    idx = L.topk_idx.cpu().numpy()
    off, perm, inv = tr.sort_slots(idx, cfg.N, capacity)
    # forward
    n = ref.norm(x, wpre, eps, 0.0)[0]
    l = n @ wr.T
    p = np.exp(l - l.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    gate = tr.gates(p, idx, True)
    xp = tr.dispatch(n, perm, k)
    g, u, h, _, _ = tr.experts_up(xp, off, wg, wu)
    y = tr.experts_down(h, off, wd)[0]
    out = tr.combine(y, gate, inv, None)[0]
    f = ref.block(out, x, wchan, "channel", wpost, wnext, eps, 0.0, scale, True)
    assert _rel(_host(L.stream), f["out"][0]) <= tol and _rel(_host(L.next), f["next"][0]) <= tol
    # backward on what is kept: exact where it is kept whole, the packed values else
    if packed:
        M = T * k
        kept_x, y = values(*L.x8, cfg.d), values(*L.y8, cfg.d)
        g, u = values(*L.g8, cfg.I), values(*L.u8, cfg.I)
        assert _rel(kept_x, n) < 0.02 and g.shape == (M, cfg.I)  # half a step in 1/64 of a block's largest
        xp, h = tr.dispatch(kept_x, perm, k), g * tr.sigmoid(g) * u
    b = ref.block_grad(r1, r2, out, f["out"][0], wchan, "channel", wpost, wnext, f["rstd_post"][0], f["rstd_next"][0], 0.0, scale, True)
    dout = b["dy"][0]
    dy, dgate, _ = tr.combine_grad(dout, y, gate, inv)
    dg, du, _, _ = tr.experts_dh(dy, g, u, off, wd)
    dl, _, _ = tr.gate_grad(p, idx, np.where(inv >= 0, dgate, 0.0), True, L.balance)
    dn = tr.combine(tr.experts_dx(dg, du, off, wg, wu)[0], None, inv, None)[0] + dl @ wr
    a = ref.block_grad(b["dresidual"][0], dn, None, x, None, "none", None, wpre, None, ref.rstd(x, eps), 0.0, 1.0, False)
    exact = {"din": a["dresidual"][0], "dw_pre": a["dw_next"][0], "dw_post": b["dw_post"][0], "dw_next": b["dw_next"][0],
             "dw_chan": b["dgate"][0], "dw_router": dl.T @ n, "dw_gate": tr.experts_dw(dg, xp, off, cfg.N)[0],
             "dw_up": tr.experts_dw(du, xp, off, cfg.N)[0], "dw_down": tr.experts_dw(h, dy, off, cfg.N)[0]}
    for name, e in exact.items():
        assert _rel(_host(getattr(L, name)), e) <= tol, name


@pytest.mark.parametrize("packed", [False, True])
def test_the_step_in_a_graph_beside_another_that_shares_the_workspace(packed):
    """Two captured steps that share one workspace, replayed in turn on one stream, give what they give alone."""
    L, x, r1, r2 = _run("granite", 64, packed)
    x2 = x.flip(0).contiguous()
    names = ["next", "din", "dw_pre", "dw_post", "dw_next", "dw_chan", "dw_gate", "dw_down"]

    def step(x):
        L.forward(x)
        L.backward(x, r2, dstream=r1)

    alone = []
    for z in (x, x2):
        step(z)
        alone.append([getattr(L, n).clone() for n in names])
    graphs = []
    for z in (x, x2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(z)
        graphs.append(g)
    for turn in (0, 1, 1, 0):
        graphs[turn].replay()
        assert all(torch.equal(getattr(L, n), a) for n, a in zip(names, alone[turn]))
    L.check()


@pytest.mark.parametrize("block,packed", [(True, False), (False, True), (True, True)])
def test_the_example_runs(block, packed):
    from train_step import train
    assert all(np.isfinite(train("tiny", 64, steps=4, block=block, packed=packed)))


@pytest.mark.parametrize("layer,T", [("tiny", 16), ("granite", 1), ("granite", 100)])
def test_block_end_behind_the_inference_layer(layer, T):
    """moe_layer_forward's float32 output into the stream and on to the next norm."""
    from expert_routing_ffn_gb300.layer import DeviceLayer, LayerBuffers, forward
    from workloads import make_tokens, make_weights
    cfg = CONFIGS[layer]
    dl = DeviceLayer(cfg, make_weights(cfg), T)
    bufs = LayerBuffers(dl, T)
    x = torch.from_numpy(make_tokens(cfg, T=T)).cuda().to(dl.dt)
    D, kind = dl.dims.with_T(T), "f32" if cfg.wtype == "f32" else "bf16"
    w = (1 + 0.2 * torch.randn(cfg.d, device="cuda")).to(dl.dt)
    n, stream, nxt = torch.empty_like(x), x.clone(), torch.empty_like(x)
    moe.moe_norm_rows(D, x, w, 1e-6, 0.0, n, None)
    forward(dl, bufs, n)
    moe.moe_block_out(D, moe.make_block(residual_scale=0.22), bufs.out[:T], stream, None, w, w, stream, nxt, None, None)
    f = ref.block(_host(bufs.out[:T]), _host(x), None, "none", _host(w), _host(w), float(np.float32(1e-6)), 0.0, float(np.float32(0.22)), True)
    for t, name in ((stream, "out"), (nxt, "next")):
        tr.check(_host(t), f[name][0], tr.rounded(*f[name], kind), name)
