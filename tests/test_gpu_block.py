"""The block's norms, gate and residual on the GPU against the plain 64-bit
implementations of block_ref, within its derived bounds."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
from test_gpu_train import TYPES, clean, empty, host, rnd, workspace
from train_ref import check, rounded

pytestmark = pytest.mark.gpu

KINDS = {"none": moe.MOE_GATE_NONE, "token": moe.MOE_GATE_TOKEN, "channel": moe.MOE_GATE_CHANNEL, "full": moe.MOE_GATE_FULL}
EPS = float(np.float32(1e-6))

# T, d, type: one value, one vector, ragged vectors, every number of threads and of vectors a thread, rows that a
# thread passes over several times, more rows than groups
SIZES = [(1, 1, "bf16"), (1, 1, "f32"), (3, 8, "bf16"), (2, 7, "f32"), (5, 100, "bf16"), (33, 256, "f32"), (33, 257, "bf16"),
         (9, 258, "bf16"), (1, 2048, "bf16"), (8, 4096, "bf16"), (4, 4097, "bf16"), (7, 1001, "f32"), (700, 64, "bf16"), (1300, 72, "f32"),
         (3, 8192, "bf16"), (2, 8192, "f32"), (3, 8200, "bf16"), (2, 9001, "f32"), (2, 20000, "bf16"), (1, 65536, "bf16"), (2, 65535, "f32"),
         (1030, 1536, "bf16"), (400, 3584, "bf16"), (257, 2050, "bf16"), (3000, 33, "f32"),
         # long batches: rows that come through shared memory, from one group of threads an SM to twelve
         (8000, 64, "bf16"), (7400, 264, "f32"), (3500, 1536, "bf16"), (1300, 3584, "bf16"), (1250, 4096, "f32"), (650, 8192, "bf16"),
         (620, 8192, "f32"), (2600, 2056, "bf16")]


def dims(T, d, kind):
    return moe.make_dims(T, d, 8, 1, 64, wtype=kind)


def strided(rng, T, d, kind, sd=1.0):
    """A tensor of token rows that are part of a wider one."""
    t, h = rnd(rng, (T, d + 24), kind, sd)
    return t[:, 8:8 + d], h[:, 8:8 + d]


def vec(rng, n, kind, sd=0.2, mean=0.0):
    t = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)) * sd + mean).to(TYPES[kind])
    return t.cuda(), t.double().numpy()


def gate_of(rng, which, T, d, kind):
    if which == "none":
        return None, None
    if which == "token":
        return vec(rng, T, "f32", 0.5, 0.3)
    if which == "channel":
        return vec(rng, d, kind, 0.5, 0.3)
    return rnd(rng, (T, d), kind, 0.5)


@pytest.mark.parametrize("T,d,kind", SIZES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_norm_and_its_gradient(T, d, kind, offset):
    rng = np.random.default_rng(T * 13 + d)
    D = dims(T, d, kind)
    x, xh = rnd(rng, (T, d), kind, 3.0)
    w, wh = vec(rng, d, kind, 0.2, 1.0 - offset)
    n, r = empty((T, d), kind), empty((T,), "f32")
    moe.moe_norm_rows(D, x, w, 1e-6, offset, n, r)
    en, on, er, orr = ref.norm(xh, wh, EPS, offset)
    check(host(n), en, rounded(en, on, kind), "n")
    check(host(r), er, rounded(er, orr, "f32"), "rstd")
    dn, dnh = rnd(rng, (T, d), kind)
    add, addh = rnd(rng, (T, d), kind)
    ws = workspace(D)
    dx, dw = empty((T, d), kind), empty((d,), "f32")
    moe.moe_norm_rows_grad(D, dn, x, r, w, offset, add, dx, dw, False, ws)
    clean(ws)
    g = ref.block_grad(addh, dnh, None, xh, None, "none", None, wh, None, host(r), offset, 1.0, False)
    check(host(dx), g["dresidual"][0], rounded(*g["dresidual"], kind), "dx")
    check(host(dw), g["dw_next"][0], rounded(*g["dw_next"], "f32"), "dw")


def _branch(rng, T, d, kind, which, y32, post, offset, wide=False):
    rows = strided if wide else lambda rng, T, d, kind, sd=1.0: rnd(rng, (T, d), kind, sd)
    y, yh = rows(rng, T, d, "f32" if y32 else kind, 2.0)
    gate, gh = gate_of(rng, which, T, d, kind)
    wp, wph = vec(rng, d, kind, 0.2, 1.0 - offset) if post else (None, None)
    wn, wnh = vec(rng, d, kind, 0.2, 1.0 - offset)
    return y, yh, gate, gh, wp, wph, wn, wnh, rows


@pytest.mark.parametrize("T,d,kind", SIZES)
@pytest.mark.parametrize("which,post,y32", [("none", True, False), ("token", True, True), ("channel", True, False), ("full", True, True),
                                            ("none", False, True), ("token", False, False), ("channel", False, True), ("full", False, False)])
def test_block_and_its_gradient(T, d, kind, which, post, y32):
    rng = np.random.default_rng(T * 17 + d + post)
    offset, scale = (1.0, 0.5) if y32 else (0.0, float(np.float32(0.22)))
    D = dims(T, d, kind)
    B = moe.make_block(1e-6, offset, scale, post, KINDS[which])
    y, yh, gate, gh, wp, wph, wn, wnh, _ = _branch(rng, T, d, kind, which, y32, post, offset)
    res, resh = rnd(rng, (T, d), kind)
    out, nxt = empty((T, d), kind), empty((T, d), kind)
    ra, rb = (empty((T,), "f32") if post else None), empty((T,), "f32")
    moe.moe_block_out(D, B, y, res, gate, wp, wn, out, nxt, ra, rb)
    f = ref.block(yh, resh, gh, which, wph, wnh, EPS, offset, scale, post)
    check(host(out), f["out"][0], rounded(*f["out"], kind), "out")
    check(host(nxt), f["next"][0], rounded(*f["next"], kind), "next")
    check(host(rb), f["rstd_next"][0], rounded(*f["rstd_next"], "f32"), "rstd_next")
    if post:
        check(host(ra), f["rstd_post"][0], rounded(*f["rstd_post"], "f32"), "rstd_post")
    # out alone
    out2 = empty((T, d), kind)
    moe.moe_block_out(D, B, y, res, gate, wp, None, out2, None, None, None)
    assert torch.equal(out2, out)

    dout, douth = rnd(rng, (T, d), kind)
    dnext, dnexth = rnd(rng, (T, d), kind)
    ws = workspace(D)
    ykind = "f32" if y32 else kind
    sums = kind if d % 3 == 0 else "f32"
    dres, dy = empty((T, d), kind), empty((T, d), ykind)
    dwp, dwn = (empty((d,), sums) if post else None), empty((d,), sums)
    dg = None if which == "none" else empty((T,), "f32") if which == "token" else empty((d,), sums) if which == "channel" else empty((T, d), kind)
    moe.moe_block_out_grad(D, B, dout, dnext, y, out, gate, wp, wn, ra, rb, dres, dy, dg, dwp, dwn, False, ws)
    clean(ws)
    g = ref.block_grad(douth, dnexth, yh, host(out), gh, which, wph, wnh, host(ra) if post else None, host(rb), offset, scale, post)
    check(host(dres), g["dresidual"][0], rounded(*g["dresidual"], kind), "dresidual")
    check(host(dy), g["dy"][0], rounded(*g["dy"], ykind), "dy")
    check(host(dwn), g["dw_next"][0], rounded(*g["dw_next"], sums), "dw_next")
    if post:
        check(host(dwp), g["dw_post"][0], rounded(*g["dw_post"], sums), "dw_post")
    if dg is not None:
        check(host(dg), g["dgate"][0], rounded(*g["dgate"], "f32" if which == "token" else sums if which == "channel" else kind), "dgate")


@pytest.mark.parametrize("T,d,kind", [(37, 264, "bf16"), (5, 1001, "f32"), (3, 10001, "bf16")])
@pytest.mark.parametrize("given", ["dout", "dnext"])
def test_either_gradient_alone_and_outputs_not_asked_for(T, d, kind, given):
    rng = np.random.default_rng(8)
    D, B = dims(T, d, kind), moe.make_block(gate=moe.MOE_GATE_CHANNEL)
    y, yh, gate, gh, wp, wph, wn, wnh, _ = _branch(rng, T, d, kind, "channel", False, True, 0.0)
    out, outh = rnd(rng, (T, d), kind)
    a, b = vec(rng, T, "f32", 0.1, 1.0), vec(rng, T, "f32", 0.1, 1.0)
    r, rh = rnd(rng, (T, d), kind)
    ws = workspace(D)
    do, dn = (r, None) if given == "dout" else (None, r)
    g = ref.block_grad(None if do is None else rh, None if dn is None else rh, yh, outh, gh, "channel", wph, wnh, a[1], b[1], 0.0, 1.0, True)
    wanted = ["dresidual", "dy", "dgate", "dw_post"] + (["dw_next"] if dn is not None else [])
    for names in [wanted] + [[n] for n in wanted]:  # all, and each alone
        t = {n: empty((T, d) if n in ("dresidual", "dy") else (d,), kind if n in ("dresidual", "dy") else "f32") for n in names}
        moe.moe_block_out_grad(D, B, do, dn, y, out, gate, wp, wn, a[0], b[0], t.get("dresidual"), t.get("dy"), t.get("dgate"),
                               t.get("dw_post"), t.get("dw_next"), False, ws)
        for n in names:
            check(host(t[n]), g[n][0], rounded(*g[n], kind if n in ("dresidual", "dy") else "f32"), n)


@pytest.mark.parametrize("T,d,kind", [(19, 256, "bf16"), (6, 100, "f32"), (4, 9000, "bf16"), (5000, 1536, "bf16")])
def test_rows_of_wider_tensors_and_results_in_place(T, d, kind):
    rng = np.random.default_rng(9)
    D, B = dims(T, d, kind), moe.make_block(gate=moe.MOE_GATE_TOKEN, residual_scale=0.5)
    y, yh, gate, gh, wp, wph, wn, wnh, rows = _branch(rng, T, d, kind, "token", False, True, 0.0, wide=True)
    res, resh = rows(rng, T, d, kind)
    frame = res.clone()
    whole = res._base.clone()
    nxt = empty((T, d + 24), kind)[:, 8:8 + d]
    ra, rb = empty((T,), "f32"), empty((T,), "f32")
    moe.moe_block_out(D, B, y, res, gate, wp, wn, res, nxt, ra, rb)  # into the residual
    f = ref.block(yh, resh, gh, "token", wph, wnh, EPS, 0.0, 0.5, True)
    check(host(res), f["out"][0], rounded(*f["out"], kind), "out")
    check(host(nxt), f["next"][0], rounded(*f["next"], kind), "next")
    whole[:, 8:8 + d] = res
    assert torch.equal(res._base, whole) and not torch.equal(frame, res)  # nothing beside the rows
    assert bool(nxt._base[:, :8].isnan().all()) and bool(nxt._base[:, 8 + d:].isnan().all())
    dout, douth = rows(rng, T, d, kind)
    dnext, dnexth = rows(rng, T, d, kind)
    dy = empty((T, d + 24), kind)[:, 8:8 + d]
    ws = workspace(D)
    g = ref.block_grad(douth, dnexth, yh, host(res), gh, "token", wph, wnh, host(ra), host(rb), 0.0, 0.5, True)
    dgate, dwn = empty((T,), "f32"), empty((d,), "f32")
    moe.moe_block_out_grad(D, B, dout, dnext, y, res, gate, wp, wn, ra, rb, dout, dy, dgate, None, dwn, False, ws)
    for name, t, k in (("dresidual", dout, kind), ("dy", dy, kind), ("dgate", dgate, "f32"), ("dw_next", dwn, "f32")):
        check(host(t), g[name][0], rounded(*g[name], k), name)
    x, xh = rows(rng, T, d, kind)
    n = empty((T, d), kind)
    moe.moe_norm_rows(D, x, None, 1e-6, 1.0, n, None)
    moe.moe_norm_rows(D, x, None, 1e-6, 1.0, x, None)  # in place
    assert torch.equal(x, n)


@pytest.mark.parametrize("d", [64, 100, 9001])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_whose_squares_pass_the_range(d, kind):
    """Rows of the type's largest values, zeros, tiny values, infinities and NaN."""
    rng = np.random.default_rng(10)
    big = float(torch.finfo(TYPES[kind]).max)
    x = torch.ones(6, d)
    x[0] = torch.from_numpy(np.where(rng.random(d) < 0.5, -big, big).astype(np.float32))
    x[1] = 0.0
    x[2] = 1e-30
    x[3, d // 2] = float("inf")
    x[4, d - 1] = float("nan")
    x = x.to(TYPES[kind]).cuda()
    D = dims(6, d, kind)
    n, r = empty((6, d), kind), empty((6,), "f32")
    moe.moe_norm_rows(D, x, None, 1e-6, 1.0, n, r)
    n, xh = host(n), host(x)
    e = ref.norm(xh[:3], None, EPS, 1.0)
    # the largest values' rstd is below float32's normal numbers: 2^-149 absolute, 2^-21 of it at 2^-128
    check(n[:3], e[0], rounded(e[0], e[1] + np.abs(e[0]) * 2.0 ** -20, kind), "n")
    assert (n[1] == 0).all()
    # an infinite row has rstd 0: zeros, and NaN in the infinite place; NaN spreads
    assert np.isnan(n[3, d // 2]) and (np.delete(n[3], d // 2) == 0).all() and np.isnan(n[4]).all() and (n[5] != 0).all()
    B = moe.make_block(post_norm=True)
    out, nxt = empty((6, d), kind), empty((6, d), kind)
    moe.moe_block_out(D, B, x, torch.zeros_like(x), None, torch.ones(d, dtype=TYPES[kind], device="cuda"),
                      torch.ones(d, dtype=TYPES[kind], device="cuda"), out, nxt, None, None)
    assert np.isfinite(host(out)[:3]).all() and np.isfinite(host(nxt)[:3]).all() and np.isnan(host(nxt)[4]).all()


@pytest.mark.parametrize("T,d", [(50, 96), (3100, 1536)])
def test_column_sums_accumulate_and_an_empty_batch_gives_zeros(T, d):
    rng = np.random.default_rng(11)
    D, B = dims(T, d, "bf16"), moe.make_block(gate=moe.MOE_GATE_CHANNEL)
    y, yh, gate, gh, wp, wph, wn, wnh, _ = _branch(rng, T, d, "bf16", "channel", False, True, 0.0)
    out, outh = rnd(rng, (T, d), "bf16")
    dout, _ = rnd(rng, (T, d), "bf16")
    a, b = vec(rng, T, "f32", 0.1, 1.0), vec(rng, T, "f32", 0.1, 1.0)
    ws = workspace(D)
    t = [empty((d,), "f32") for _ in range(3)]
    run = lambda acc, D=D, T=T: moe.moe_block_out_grad(D, B, dout[:T], dout[:T], y[:T], out[:T], gate, wp, wn, a[0][:T], b[0][:T], None, None,  # noqa: E731
                                                       t[0], t[1], t[2], acc, ws)
    run(False)
    once = [v.clone() for v in t]
    run(True)
    assert all(torch.equal(v, 2 * o) for v, o in zip(t, once))
    none = dims(0, d, "bf16")
    run(True, none, 0)
    assert all(torch.equal(v, 2 * o) for v, o in zip(t, once))
    run(False, none, 0)
    assert not any(bool(v.any()) for v in t)
    e = torch.zeros((0, d), dtype=torch.bfloat16, device="cuda")
    moe.moe_norm_rows(none, e, None, 1e-6, 1.0, e, None)
    moe.moe_block_out(none, B, e, e, gate, wp, wn, e, e, None, None)
    dw = empty((d,), "bf16")
    moe.moe_norm_rows_grad(none, e, e, a[0], wn, 0.0, None, e, dw, False, ws)
    assert not dw.any()


@pytest.mark.parametrize("T", [300, 5000])
def test_repeats_bit_for_bit_in_a_graph_and_on_another_stream(T):
    """Captured together, replayed on new values, and run on a stream of their own; the order of the sums is fixed."""
    rng = np.random.default_rng(12)
    d = 1536
    D, B = dims(T, d, "bf16"), moe.make_block(gate=moe.MOE_GATE_TOKEN, residual_scale=0.22)
    y, _, gate, _, wp, _, wn, _, _ = _branch(rng, T, d, "bf16", "token", True, True, 0.0)
    res, dout, dnext = (rnd(rng, (T, d), "bf16")[0] for _ in range(3))
    ws = workspace(D)
    f = [empty((T, d), "bf16"), empty((T, d), "bf16"), empty((T,), "f32"), empty((T,), "f32")]
    g = [empty((T, d), "bf16"), empty((T, d), "f32"), empty((T,), "f32"), empty((d,), "f32"), empty((d,), "f32")]

    def both():
        moe.moe_block_out(D, B, y, res, gate, wp, wn, *f)
        moe.moe_block_out_grad(D, B, dout, dnext, y, f[0], gate, wp, wn, f[2], f[3], *g, False, ws)

    both()
    first = [t.clone() for t in f + g]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, f + g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    new = rnd(rng, (T, d), "bf16")[0]
    res.copy_(new)
    graph.replay()
    replayed = [t.clone() for t in f + g]
    both()
    assert all(torch.equal(a, b) for a, b in zip(replayed, f + g)) and not torch.equal(first[0], f[0])
