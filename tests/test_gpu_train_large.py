"""The training step's kernels where sizes turn over: tensors of more than
2^31 elements, more experts than 256, tiles of exactly one unit, one tile and
one row more."""
import numpy as np
import pytest
import torch

import expert_routing_ffn_gb300 as moe
import train_ref as ref
from test_gpu_train import Ffn, clean, empty, host, workspace

pytestmark = pytest.mark.gpu

EDGES = [  # T, d, N, k, I, routing, type
    (32, 64, 2, 1, 64, "one", "bf16"), (33, 64, 2, 1, 64, "one", "bf16"), (64, 192, 3, 1, 128, "one", "bf16"),
    (65, 192, 3, 1, 128, "one", "bf16"), (256, 128, 3, 1, 192, "one", "bf16"), (257, 128, 3, 1, 192, "one", "bf16"),
    (600, 64, 300, 8, 72, "skew", "bf16"), (513, 264, 512, 4, 64, "some", "bf16"), (2000, 512, 8, 2, 512, "skew", "bf16"),
    (90, 64, 300, 2, 40, "some", "f32"), (17, 8, 4, 2, 8, "all", "bf16"),
]


@pytest.mark.parametrize("case", EDGES, ids=lambda c: "-".join(map(str, c)))
def test_every_product_at_the_edges(case):
    f = Ffn(*case)
    (dg, dgh), (du, duh), (dy, dyh), (hq, hh) = f.rows(f.I), f.rows(f.I), f.rows(f.d), f.rows(f.I)
    g, u, h = (empty((f.M, f.I), f.kind) for _ in range(3))
    moe.moe_experts_up(f.D, f.x, f.doff, f.wg, f.wu, g, u, h, f.ws)
    eg, eu, eh, mg, mu = ref.experts_up(f.xh, f.off, f.wgh, f.wuh)
    ref.check(host(g), eg, ref.bound(eg, f.d, mg, f.kind), "g")
    ref.check(host(u), eu, ref.bound(eu, f.d, mu, f.kind), "u")
    ref.check(host(h), eh, ref.up_h_limit(eg, eu, eh, mg, mu, f.d, f.kind), "h")
    y = empty((f.M, f.d), f.kind)
    moe.moe_experts_down(f.D, hq, f.doff, f.wd, y, f.ws)
    ey, mag = ref.experts_down(hh, f.off, f.wdh)
    ref.check(host(y), ey, ref.bound(ey, f.I, mag, f.kind), "y")
    dx, dwg, dwu = empty((f.M, f.d), f.kind), empty((f.N, f.I, f.d), f.kind), empty((f.N, f.I, f.d), f.kind)
    moe.moe_experts_up_grad(f.D, dg, du, f.x, f.doff, f.wg, f.wu, dx, dwg, dwu, False, f.ws)
    edx, mag = ref.experts_dx(dgh, duh, f.off, f.wgh, f.wuh)
    ref.check(host(dx), edx, ref.bound(edx, 2 * f.I, mag, f.kind), "dx")
    for name, got, a in (("dw_gate", dwg, dgh), ("dw_up", dwu, duh)):
        e, mag, n = ref.experts_dw(a, f.xh, f.off, f.N)
        ref.check(host(got), e, ref.bound(e, n, mag, f.kind), name)
    odg, odu, dwd = empty((f.M, f.I), f.kind), empty((f.M, f.I), f.kind), empty((f.N, f.I, f.d), "f32")
    gq, uq = torch.nan_to_num(dg), torch.nan_to_num(du)
    moe.moe_experts_down_grad(f.D, dy, hq, gq, uq, f.doff, f.wd, odg, odu, dwd, False, f.ws)
    f.done()
    edg, edu, og, ou = ref.experts_dh(dyh, dgh, duh, f.off, f.wdh)
    ref.check(host(odg), edg, ref.rounded(edg, og, f.kind), "dg")
    ref.check(host(odu), edu, ref.rounded(edu, ou, f.kind), "du")
    e, mag, n = ref.experts_dw(hh, dyh, f.off, f.N)
    ref.check(host(dwd), e, ref.bound(e, n, mag, "f32"), "dw_down")


def test_rows_beyond_2_to_31_elements():
    """dispatch, combine and both gradients on 560000 grouped rows of 4096."""
    T, d, N, k = 70000, 4096, 8, 8
    D = moe.make_dims(T, d, N, k, 64, wtype="bf16")
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda").normal_()
    idx = torch.arange(N, dtype=torch.int32, device="cuda").repeat(T, 1).contiguous()
    ws, xp = workspace(D), torch.empty((T * k, d), dtype=torch.bfloat16, device="cuda")
    off, perm, inv = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (N + 1, T * k, T * k))
    moe.moe_dispatch_rows(D, x, idx, 0, xp, off, perm, inv, ws)
    clean(ws)
    assert off.tolist() == [e * T for e in range(N + 1)]
    for e in (0, N - 1):  # expert e has every token in order
        assert torch.equal(xp[e * T:(e + 1) * T], x)
    gate = torch.zeros((T, k), device="cuda")
    gate[:, N - 1] = 1.0
    out, dgate = torch.empty_like(x), torch.empty((T, k), device="cuda")
    moe.moe_combine_rows(D, xp, gate, inv, None, out)
    assert torch.equal(out, x)
    dy = torch.empty_like(xp)
    moe.moe_combine_rows_grad(D, x, xp, gate, inv, dy, dgate)
    assert torch.equal(dy[-T:], x) and not dy[:T].any()
    assert torch.equal(dgate[:, 0], dgate[:, N - 1])
    dot = x[-1].double().square().sum()
    assert abs(float(dgate[-1, -1] - dot)) <= float(dot) * d * ref.STEP


def test_products_beyond_2_to_31_elements():
    """560000 rows on 4096 columns: the last expert's rows lie past 2^31."""
    T, d, N, k, I = 70000, 4096, 8, 8, 64
    D = moe.make_dims(T, d, N, k, I, wtype="bf16")
    off = torch.arange(N + 1, dtype=torch.int32, device="cuda") * T
    h = torch.empty((T * k, I), dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.empty((N, I, d), dtype=torch.bfloat16, device="cuda").normal_(0, 0.1)
    y, ws = torch.full((T * k, d), float("nan"), dtype=torch.bfloat16, device="cuda"), workspace(D)
    moe.moe_experts_down(D, h, off, w, y, ws)
    dw = torch.empty((N, I, d), device="cuda")
    moe.moe_experts_down_grad(D, y, h, None, None, off, w, None, None, dw, False, ws)
    clean(ws)
    assert not torch.isnan(y).any()
    rows = [0, T * k // 2, T * k - 1]
    exact = np.stack([host(h[r]) @ host(w[r // T]) for r in rows])
    mag = np.stack([np.abs(host(h[r])) @ np.abs(host(w[r // T])) for r in rows])
    ref.check(np.stack([host(y[r]) for r in rows]), exact, ref.bound(exact, I, mag, "bf16"), "y")
    last = slice((N - 1) * T, N * T)
    e = (h[last].double().T @ y[last][:, -64:].double()).cpu().numpy()
    m = (h[last].double().abs().T @ y[last][:, -64:].double().abs()).cpu().numpy()
    ref.check(host(dw[-1])[:, -64:], e, ref.bound(e, T, m, "f32"), "dw")


def _at_the_end(t):
    """The same tensor as the last rows of a buffer that fills its allocation."""
    n = t.numel() * t.element_size()
    buf = torch.empty((n + (12 << 20)) // (2 << 20) * (2 << 20), dtype=torch.uint8, device="cuda")
    view = buf[buf.numel() - n:].view(t.dtype).view(t.shape)
    return view.copy_(t)


@pytest.mark.parametrize("T,d,N,k,I", [(48, 1536, 40, 8, 512), (600, 512, 8, 2, 1024)])
def test_rows_that_end_with_their_allocation(T, d, N, k, I):
    """Small segments of large row tensors: nothing past the last row is read, and the results are
    those of rows with others behind them."""
    torch.cuda.empty_cache()
    f = Ffn(T, d, N, k, I, "all", "bf16")
    (dg, _), (du, _), (dy, _), (h, _), (g, _), (u, _) = (f.rows(n) for n in (I, I, d, I, I, I))
    rows = [torch.nan_to_num(t) for t in (f.x, dg, du, dy, h, g, u)]

    def step(x, dg, du, dy, h, g, u, end):
        place = _at_the_end if end else (lambda t: t)
        outs = [place(empty((f.M, n), "bf16")) for n in (I, I, I, d, d, I, I)]
        dws = [empty((N, I, d), "f32") for _ in range(3)]
        moe.moe_experts_up(f.D, x, f.doff, f.wg, f.wu, *outs[:3], f.ws)
        moe.moe_experts_down(f.D, h, f.doff, f.wd, outs[3], f.ws)
        moe.moe_experts_up_grad(f.D, dg, du, x, f.doff, f.wg, f.wu, outs[4], dws[0], dws[1], False, f.ws)
        moe.moe_experts_down_grad(f.D, dy, h, g, u, f.doff, f.wd, outs[5], outs[6], dws[2], False, f.ws)
        f.done()
        return outs + dws

    for a, b in zip(step(*rows, False), step(*[_at_the_end(t) for t in rows], True)):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))
