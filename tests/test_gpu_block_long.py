"""Norms and blocks of long batches, whose rows come through shared memory: every
call at lengths where it takes that form (four rows and more for every group of
threads), with inputs and outputs left out, and with rows out of range among
the others."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
from test_gpu_block import EPS, KINDS, _branch, dims, vec
from test_gpu_train import TYPES, clean, empty, host, rnd, workspace
from train_ref import check, rounded

pytestmark = pytest.mark.gpu

# d, type, the most groups an SM has of any of the calls: groups of two warps, of three, of seven; float32 with four
# vectors a thread, all of them and a part
SHAPES = [(520, "bf16", 12), (1536, "bf16", 8), (3584, "bf16", 3), (4096, "f32", 3), (2056, "f32", 4)]


def tokens(most):
    return 4 * torch.cuda.get_device_properties(0).multi_processor_count * most + 5


@pytest.mark.parametrize("d,kind,most", SHAPES)
@pytest.mark.parametrize("weighted,added,offset,gkind", [(True, True, 0.0, "f32"), (True, False, 1.0, "layer"), (False, False, 1.0, "f32")])
def test_norm_and_its_gradient(d, kind, most, weighted, added, offset, gkind):
    T, rng = tokens(most), np.random.default_rng(d)
    D = dims(T, d, kind)
    x, xh = rnd(rng, (T, d), kind, 3.0)
    w, wh = vec(rng, d, kind, 0.2, 1.0 - offset) if weighted else (None, None)
    n, r = empty((T, d), kind), empty((T,), "f32")
    moe.moe_norm_rows(D, x, w, 1e-6, offset, n, r)
    en, on, er, orr = ref.norm(xh, wh, EPS, offset)
    check(host(n), en, rounded(en, on, kind), "n")
    check(host(r), er, rounded(er, orr, "f32"), "rstd")
    dn, dnh = rnd(rng, (T, d), kind)
    add, addh = rnd(rng, (T, d), kind) if added else (None, None)
    ws, gk = workspace(D), kind if gkind == "layer" else "f32"
    dx, dw = empty((T, d), kind), empty((d,), gk)
    moe.moe_norm_rows_grad(D, dn, x, r, w, offset, add, dx, dw, False, ws)
    clean(ws)
    g = ref.block_grad(addh, dnh, None, xh, None, "none", None, wh, None, host(r), offset, 1.0, False)
    check(host(dx), g["dresidual"][0], rounded(*g["dresidual"], kind), "dx")
    check(host(dw), g["dw_next"][0], rounded(*g["dw_next"], gk), "dw")
    dx2 = empty((T, d), kind)
    moe.moe_norm_rows_grad(D, dn, x, r, w, offset, add, dx2, None, False, ws)
    assert torch.equal(dx2, dx)


@pytest.mark.parametrize("d,kind,most", SHAPES)
@pytest.mark.parametrize("which,post,y32", [("none", True, True), ("token", True, False), ("channel", False, False), ("full", True, True)])
def test_block_forward(d, kind, most, which, post, y32):
    T, rng = tokens(most), np.random.default_rng(d + 1)
    D, B = dims(T, d, kind), moe.make_block(1e-6, 0.0, 0.5, post, KINDS[which])
    y, yh, gate, gh, wp, wph, wn, wnh, _ = _branch(rng, T, d, kind, which, y32, post, 0.0)
    res, resh = rnd(rng, (T, d), kind)
    out, nxt, rb = empty((T, d), kind), empty((T, d), kind), empty((T,), "f32")
    ra = empty((T,), "f32") if post else None
    moe.moe_block_out(D, B, y, res, gate, wp, wn, out, nxt, ra, rb)
    f = ref.block(yh, resh, gh, which, wph, wnh, EPS, 0.0, 0.5, post)
    check(host(out), f["out"][0], rounded(*f["out"], kind), "out")
    check(host(nxt), f["next"][0], rounded(*f["next"], kind), "next")
    check(host(rb), f["rstd_next"][0], rounded(*f["rstd_next"], "f32"), "rstd_next")
    if post:
        check(host(ra), f["rstd_post"][0], rounded(*f["rstd_post"], "f32"), "rstd_post")
    out2 = empty((T, d), kind)
    moe.moe_block_out(D, B, y, res, gate, wp, None, out2, None, None, None)
    assert torch.equal(out2, out)


@pytest.mark.parametrize("d,kind,most", [(1536, "bf16", 5), (4096, "f32", 2)])
@pytest.mark.parametrize("which", ["channel", "full"])
@pytest.mark.parametrize("given", ["dout", "dnext"])
def test_either_gradient_alone_and_outputs_not_asked_for(d, kind, most, which, given):
    T, rng = tokens(most), np.random.default_rng(d + 2)
    D, B = dims(T, d, kind), moe.make_block(gate=KINDS[which])
    y, yh, gate, gh, wp, wph, wn, wnh, _ = _branch(rng, T, d, kind, which, False, True, 0.0)
    out, outh = rnd(rng, (T, d), kind)
    a, b = vec(rng, T, "f32", 0.1, 1.0), vec(rng, T, "f32", 0.1, 1.0)
    r, rh = rnd(rng, (T, d), kind)
    ws = workspace(D)
    do, dn = (r, None) if given == "dout" else (None, r)
    g = ref.block_grad(None if do is None else rh, None if dn is None else rh, yh, outh, gh, which, wph, wnh, a[1], b[1], 0.0, 1.0, True)
    wide = ("dresidual", "dy") + (("dgate",) if which == "full" else ())
    wanted = ["dresidual", "dy", "dgate", "dw_post"] + (["dw_next"] if dn is not None else [])
    for names in [wanted] + [[n] for n in wanted]:  # all, and each alone
        t = {n: empty((T, d) if n in wide else (d,), kind if n in wide else "f32") for n in names}
        moe.moe_block_out_grad(D, B, do, dn, y, out, gate, wp, wn, a[0], b[0], t.get("dresidual"), t.get("dy"), t.get("dgate"),
                               t.get("dw_post"), t.get("dw_next"), False, ws)
        clean(ws)
        for n in names:
            check(host(t[n]), g[n][0], rounded(*g[n], kind if n in wide else "f32"), n)


def _out_of_range(rng, T, d, kind, n_kinds):
    """Rows of the type's largest values, zeros, tiny values, an infinity, a NaN, each some times among ordinary ones:
    (ordinary rows, the same with those among them, their numbers by kind)."""
    t, _ = rnd(rng, (T, d), kind)
    x, big = t.clone(), float(torch.finfo(TYPES[kind]).max)
    at = np.sort(rng.permutation(T)[:n_kinds * 6].reshape(n_kinds, 6), 1)
    signs = torch.from_numpy(np.where(rng.random((6, d)) < 0.5, -big, big).astype(np.float32)).to(TYPES[kind]).cuda()
    rows = [torch.from_numpy(a).cuda() for a in at]
    x[rows[0]] = signs
    x[rows[1]] = 0.0
    x[rows[2]] = 1e-30
    x[rows[3], d // 2] = float("inf")
    x[rows[4], d - 1] = float("nan")
    return t, x, at


@pytest.mark.parametrize("d,kind,most", SHAPES)
def test_rows_out_of_range_among_others(d, kind, most):
    T, rng = tokens(most), np.random.default_rng(d + 3)
    D = dims(T, d, kind)
    t, x, at = _out_of_range(rng, T, d, kind, 5)
    rest = np.setdiff1d(np.arange(T), at.reshape(-1))
    rows = torch.from_numpy(rest).cuda()
    w, wh = vec(rng, d, kind, 0.2, 1.0)

    def norm(x):
        n, r = empty((T, d), kind), empty((T,), "f32")
        moe.moe_norm_rows(D, x, w, 1e-6, 0.0, n, r)
        return n, r

    def grad(x, r, ws):
        dx, dw = empty((T, d), kind), empty((d,), "f32")
        moe.moe_norm_rows_grad(D, t, x, r, w, 0.0, t, dx, dw, False, ws)
        clean(ws)
        return dx, dw

    (n0, r0), (n, r) = norm(t), norm(x)
    assert torch.equal(n[rows], n0[rows]) and torch.equal(r[rows], r0[rows])  # the others do not notice
    nh, xh = host(n), host(x)
    finite = at[:3].reshape(-1)
    e, off, _, _ = ref.norm(xh[finite], wh, EPS, 0.0)
    # the largest values' rstd is below float32's normal numbers: 2^-149 absolute, 2^-21 of it at 2^-128
    check(nh[finite], e, rounded(e, off + np.abs(e) * 2.0 ** -20, kind), "n")
    assert (nh[at[1]] == 0).all() and np.isnan(nh[at[4]]).all()
    assert np.isnan(nh[at[3], d // 2]).all() and (np.delete(nh[at[3]], d // 2, 1) == 0).all()
    ws = workspace(D)
    (dx0, _), (dx, dw) = grad(t, r0, ws), grad(x, r, ws)
    assert torch.equal(dx[rows], dx0[rows]) and bool(dw.isnan().any())
    assert bool(dx[torch.from_numpy(finite).cuda()].isfinite().all()) and bool(dx[torch.from_numpy(at[4]).cuda()].isnan().all())


@pytest.mark.parametrize("d,kind,most", SHAPES)
@pytest.mark.parametrize("where", ["branch", "residual"])
def test_rows_out_of_range_in_a_block(d, kind, most, where):
    """In the branch the first of a row's two sums passes the range, in the residual the second."""
    T, rng = tokens(most), np.random.default_rng(d + 4)
    D, B = dims(T, d, kind), moe.make_block(gate=moe.MOE_GATE_TOKEN, residual_scale=0.25)
    t, x, at = _out_of_range(rng, T, d, kind, 5)
    rest = torch.from_numpy(np.setdiff1d(np.arange(T), at.reshape(-1))).cuda()
    other, otherh = rnd(rng, (T, d), kind)
    w, wh = vec(rng, d, kind, 0.2, 1.0)
    gate, gh = vec(rng, T, "f32", 0.1, 1.0)

    def run(x):
        o = empty((T, d), kind), empty((T, d), kind), empty((T,), "f32"), empty((T,), "f32")
        y, res = (x, other) if where == "branch" else (other, x)
        moe.moe_block_out(D, B, y, res, gate, w, w, *o)
        return o

    clean_run, o = run(t), run(x)
    assert all(torch.equal(a[rest], b[rest]) for a, b in zip(o, clean_run))
    out, nxt, xh = host(o[0]), host(o[1]), host(x)
    finite = at[:3].reshape(-1)
    if where == "residual":  # a half of the largest values, so that the branch does not carry them out of range
        x[torch.from_numpy(at[0]).cuda()] *= 0.5
        o, xh = run(x), host(x)
        out, nxt = host(o[0]), host(o[1])
    f = ref.block(*((xh[finite], otherh[finite]) if where == "branch" else (otherh[finite], xh[finite])), gh[finite], "token", wh, wh, EPS,
                  0.0, 0.25, True)
    for name, got in (("out", out), ("next", nxt)):
        e, off = f[name]
        check(got[finite], e, rounded(e, off + np.abs(f["out"][0] - (otherh if where == "branch" else xh)[finite]) * 2.0 ** -20 +
                                      np.abs(e) * 2.0 ** -20, kind), name)
    # an infinity in the branch has rstd 0 and leaves NaN in its place of out, so next is NaN; in the residual it stays
    # one, and next has zeros beside it
    assert np.isnan(nxt[at[4]]).all() and np.isnan(nxt[at[3], d // 2]).all()
    beside = np.delete(nxt[at[3]], d // 2, 1)
    assert np.isnan(beside).all() if where == "branch" else (beside == 0).all()
    assert np.isnan(out[at[4], d - 1]).all() and not np.isfinite(out[at[3], d // 2]).any()
