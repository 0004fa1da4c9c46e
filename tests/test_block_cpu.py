"""The block's norms and the packed activations without a GPU: the gradients'
formulas against central differences of the forward formulas (64 bits), the
packed format's plain implementation, the calls' refusals, sizes and devices."""
import ctypes as C

import numpy as np
import pytest

import block_ref as ref
import expert_routing_ffn_gb300 as moe
from test_train_cpu import BASE, DIFF_TOL, _slope


@pytest.mark.parametrize("kind", ref.GATES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_block_gradient_formula_matches_differences(kind, post, offset):
    rng = np.random.default_rng(3)
    T, d, eps, scale = 4, 7, 1e-3, 0.7
    y, res = rng.normal(size=(T, d)), rng.normal(size=(T, d))
    gate = {"none": None, "token": rng.normal(size=T), "channel": rng.normal(size=d), "full": rng.normal(size=(T, d))}[kind]
    wp, wn = (rng.normal(size=d) if post else None), rng.normal(size=d)
    r1, r2 = rng.normal(size=(T, d)), rng.normal(size=(T, d))

    def loss(y, res, gate, wp, wn):
        f = ref.block(y, res, gate, kind, wp, wn, eps, offset, scale, post)
        return float((r1 * f["out"][0]).sum() + (r2 * f["next"][0]).sum())

    at = [y, res, gate, wp, wn]
    f = ref.block(*at[:3], kind, *at[3:], eps, offset, scale, post)
    a = f["rstd_post"][0] if post else None
    g = ref.block_grad(r1, r2, y, f["out"][0], gate, kind, wp, wn, a, f["rstd_next"][0], offset, scale, post)
    for i, name in enumerate(("dy", "dresidual", "dgate", "dw_post", "dw_next")):
        if at[i] is None:
            assert name not in g
            continue
        v = rng.normal(size=at[i].shape)
        s = _slope(lambda z: loss(*[z if j == i else at[j] for j in range(5)]), at[i], v)
        assert abs(s - float((g[name][0] * v).sum())) <= DIFF_TOL * max(1.0, abs(s)), name


def test_norm_gradient_is_the_block_gradient_without_a_branch():
    rng = np.random.default_rng(4)
    x, w, r, add = (rng.normal(size=s) for s in ((3, 9), (9,), (3, 9), (3, 9)))
    f = lambda x, w: float((r * ref.norm(x, w, 1e-3, 0.0)[0]).sum() + (add * x).sum())  # noqa: E731
    g = ref.block_grad(add, r, None, x, None, "none", None, w, None, ref.rstd(x, 1e-3), 0.0, 1.0, False)
    for name, i in (("dresidual", 0), ("dw_next", 1)):
        v = rng.normal(size=(x, w)[i].shape)
        s = _slope(lambda z: f(*[z if j == i else (x, w)[j] for j in range(2)]), (x, w)[i], v)
        assert abs(s - float((g[name][0] * v).sum())) <= DIFF_TOL * max(1.0, abs(s))


def test_packed_values_are_within_half_a_step_and_a_127th_of_the_largest():
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((7, 101)) * 10.0 ** rng.integers(-30, 30, (7, 1))).astype(np.float32).astype(np.float64)
    x[3, 40:50] = 0.0
    q, E = ref.pack(x)
    v = ref.unpack(q, E, 101)
    pad = np.zeros((7, 4 * 32))
    pad[:, :101] = np.abs(x - v)
    off, big = pad.reshape(7, 4, 32).max(2), np.zeros((7, 4 * 32))
    big[:, :101] = np.abs(x)
    big = big.reshape(7, 4, 32).max(2)
    assert np.abs(q).max() == 127 and (off <= 0.5 * 2.0 ** (E - 127.0)).all() and (off <= big / 127).all()
    assert (q.reshape(7, -1)[:, 101:] == 0).all()
    assert np.array_equal(ref.columns(ref.kept(q), 4), q)


# ---------------------------------------------------------------- refusals

A, WS = 0x10000, 1 << 20  # addresses that a refused call never follows


def _block(**kw):
    return moe.make_block(**kw)


def _calls(D, null=None, ws=WS, n=16 << 20, ld=0, g=moe.MOE_DTYPE_BF16, acc=0, odd=None, block=None, yt=None, eps=1e-6, offset=0.0,
           rows=4, cols=40, div=1):
    L, r = moe.lib(), C.byref(D)
    yt = D.wtype if yt is None else yt
    b = None if null == "block" else C.byref(block if block is not None else _block(gate=moe.MOE_GATE_TOKEN))

    def a(name, v=A):
        return None if null == name else v + 1 if odd == name else v

    return {
        "norm": lambda: L.moe_norm_rows(r, a("x"), ld, a("w"), eps, offset, a("n"), ld, a("rstd"), None),
        "norm_grad": lambda: L.moe_norm_rows_grad(r, a("dn"), ld, a("x"), ld, a("rstd"), a("w"), offset, a("add"), ld,
                                                  a("dx"), ld, a("dw"), g, acc, ws, n, None),
        "block": lambda: L.moe_block_out(r, b, a("y"), ld, yt, a("res"), ld, a("gate"), a("w_post"), a("w_next"), a("out"), ld,
                                         a("next"), ld, a("rstd_post"), a("rstd_next"), None),
        "block_grad": lambda: L.moe_block_out_grad(r, b, a("dout"), ld, a("dnext"), ld, a("y"), ld, yt, a("out"), ld, a("gate"),
                                                   a("w_post"), a("w_next"), a("rstd_post"), a("rstd_next"), a("dres"), ld,
                                                   a("dy"), ld, a("dgate"), a("dw_post"), a("dw_next"), g, acc, ws, n, None),
        "pack": lambda: L.moe_pack_rows(rows, cols, a("x"), ld, g, a("q"), a("scale"), None),
        "unpack": lambda: L.moe_unpack_rows(rows, cols, a("q"), a("scale"), a("index"), div, rows, a("out"), ld, g, None),
        "up": lambda: L.moe_experts_up_packed(r, a("x_perm"), a("off"), a("wg"), a("wu"), a("g_q"), a("g_scale"), a("u_q"),
                                              a("u_scale"), a("h"), ws, n, None),
        "down_grad": lambda: L.moe_experts_down_grad_packed(r, a("dy"), a("g_q"), a("g_scale"), a("u_q"), a("u_scale"), a("off"),
                                                            a("wd"), a("h"), a("dg"), a("du"), a("dwd"), g, acc, ws, n, None),
        "combine_grad": lambda: L.moe_combine_rows_grad_packed(r, a("dout"), ld, a("y_q"), a("y_scale"), a("gate"), a("inv"),
                                                               a("dy"), a("dgate"), None),
    }


DIMS_CALLS = ("norm", "norm_grad", "block", "block_grad", "up", "down_grad", "combine_grad")


@pytest.mark.parametrize("kw,status", [
    (dict(N=513), moe.MOE_ERR_UNSUPPORTED), (dict(k=17, N=32), moe.MOE_ERR_UNSUPPORTED), (dict(T=1 << 24, k=2), moe.MOE_ERR_UNSUPPORTED),
    (dict(d=1 << 17), moe.MOE_ERR_UNSUPPORTED), (dict(T=-1), moe.MOE_ERR_INVALID_ARG), (dict(d=0), moe.MOE_ERR_INVALID_ARG),
])
@pytest.mark.parametrize("call", DIMS_CALLS)
def test_bad_dims_are_refused(call, kw, status):
    assert _calls(moe.make_dims(**dict(BASE, **kw)))[call]() == status


REQUIRED = [("norm", n) for n in ("x", "n")] + [("norm_grad", n) for n in ("dn", "x", "rstd", "dx")] + \
    [("block", n) for n in ("block", "y", "res", "gate", "out")] + \
    [("block", "next")] + \
    [("block_grad", n) for n in ("block", "y", "out", "gate", "rstd_post", "rstd_next")] + \
    [("block_grad", "dnext")] + \
    [("pack", n) for n in ("x", "q", "scale")] + [("unpack", n) for n in ("q", "scale", "out")] + \
    [("up", n) for n in ("x_perm", "off", "wg", "wu", "g_q", "g_scale", "u_q", "u_scale", "h")] + \
    [("down_grad", n) for n in ("dy", "g_q", "g_scale", "u_q", "u_scale", "off", "wd", "h", "dg", "du")] + \
    [("combine_grad", n) for n in ("dout", "inv", "y_q", "y_scale")]


@pytest.mark.parametrize("call,arg", REQUIRED)
def test_missing_buffers_are_refused_before_cuda(call, arg):
    """("block", "next") and ("block_grad", "dnext"): their norm's weight, rstd and gradient are then given for nothing."""
    assert _calls(moe.make_dims(**BASE), null=arg)[call]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call,arg", [(c, n) for c, names in {
    "norm": ("x", "w", "n", "rstd"), "norm_grad": ("dn", "x", "w", "add", "dx", "dw", "rstd"),
    "block": ("y", "res", "gate", "w_post", "w_next", "out", "next", "rstd_post", "rstd_next"),
    "block_grad": ("dout", "dnext", "y", "out", "gate", "w_post", "w_next", "rstd_post", "rstd_next", "dres", "dy", "dgate",
                   "dw_post", "dw_next"),
    "pack": ("x", "q"), "unpack": ("q", "index", "out"), "up": ("x_perm", "off", "g_q", "u_q", "h"),
    "down_grad": ("dy", "g_q", "off", "wd", "h", "dg", "dwd"), "combine_grad": ("dout", "y_q", "gate", "inv", "dy", "dgate"),
}.items() for n in names])
def test_misaligned_buffers_are_refused(call, arg):
    assert _calls(moe.make_dims(**BASE), odd=arg)[call]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kind", [moe.MOE_GATE_CHANNEL, moe.MOE_GATE_FULL])
def test_other_gates_are_checked_too(kind):
    b, D = _block(gate=kind), moe.make_dims(**BASE)
    for call in ("block", "block_grad"):
        assert _calls(D, block=b, null="gate")[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, block=b, odd="gate")[call]() == moe.MOE_ERR_INVALID_ARG
    assert _calls(D, block=b, odd="dgate")["block_grad"]() == moe.MOE_ERR_INVALID_ARG


def test_strides_numbers_types_and_workspaces():
    D, bad = moe.make_dims(**BASE), float("nan")
    for call in ("norm", "norm_grad", "block", "block_grad", "combine_grad"):
        assert _calls(D, ld=39)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, ld=-64)[call]() == moe.MOE_ERR_INVALID_ARG
    for eps in (0.0, -1e-6, bad, float("inf")):
        assert _calls(D, eps=eps)["norm"]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, block=_block(eps=eps, gate=moe.MOE_GATE_TOKEN))["block"]() == moe.MOE_ERR_INVALID_ARG
    for kw in (dict(weight_offset=bad), dict(residual_scale=float("inf")), dict(gate=4), dict(gate=-1), dict(gate=moe.MOE_GATE_NONE),
               dict(gate=moe.MOE_GATE_TOKEN, post_norm=False)):
        # a gate with MOE_GATE_NONE, a norm's weight without the norm
        for call in ("block", "block_grad"):
            assert _calls(D, block=_block(**kw))[call]() == moe.MOE_ERR_INVALID_ARG, kw
    for call in ("norm", "norm_grad"):
        assert _calls(D, offset=bad)[call]() == moe.MOE_ERR_INVALID_ARG
    for call in ("block", "block_grad"):
        assert _calls(D, yt=7)[call]() == moe.MOE_ERR_UNSUPPORTED
        assert _calls(moe.make_dims(**dict(BASE, wtype="f32")), yt=moe.MOE_DTYPE_BF16, g=moe.MOE_DTYPE_F32)[call]() == moe.MOE_ERR_UNSUPPORTED
    need = moe.moe_train_workspace_size(D)
    for call in ("norm_grad", "block_grad", "up", "down_grad"):
        assert _calls(D, ws=None)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, ws=WS + 8)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, n=100)[call]() == moe.MOE_ERR_CAPACITY
    wide = moe.make_dims(**dict(BASE, T=4096, d=4096))
    for call in ("norm_grad", "block_grad"):
        assert _calls(wide, n=need)[call]() == moe.MOE_ERR_CAPACITY
    for call in ("norm_grad", "block_grad", "down_grad"):
        assert _calls(D, acc=1)[call]() == moe.MOE_ERR_UNSUPPORTED  # accumulation into bf16
        assert _calls(D, g=7)[call]() == moe.MOE_ERR_UNSUPPORTED
    # one of the two gradients is needed
    L, r = moe.lib(), C.byref(D)
    b = C.byref(_block())
    assert L.moe_block_out_grad(r, b, None, 0, None, 0, A, 0, D.wtype, A, 0, None, None, None, A, A, A, 0, A, 0, None, None, None,
                                D.wtype, 0, WS, 16 << 20, None) == moe.MOE_ERR_INVALID_ARG


def test_packed_sizes_and_limits():
    assert moe.moe_packed_size(3, 33) == (3 * 64, 3 * 2)
    assert moe.moe_packed_size(0, 1) == (0, 0)
    D = moe.make_dims(**BASE)
    for kw, status in ((dict(rows=-1), moe.MOE_ERR_INVALID_ARG), (dict(cols=0), moe.MOE_ERR_INVALID_ARG),
                       (dict(rows=(1 << 24) + 1), moe.MOE_ERR_UNSUPPORTED), (dict(cols=65537), moe.MOE_ERR_UNSUPPORTED),
                       (dict(ld=39), moe.MOE_ERR_INVALID_ARG), (dict(g=7), moe.MOE_ERR_UNSUPPORTED)):
        for call in ("pack", "unpack"):
            assert _calls(D, **kw)[call]() == status, (call, kw)
    assert _calls(D, div=0)["unpack"]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("dims", [BASE, dict(BASE, T=0), dict(BASE, T=1 << 23), dict(BASE, T=1 << 20, d=65536), dict(BASE, T=1000, d=65536, N=512, k=16)])
def test_workspace_stays_below_its_documented_limit(dims):
    assert 0 < moe.moe_train_workspace_size(moe.make_dims(**dims)) <= 16 << 20


def test_calls_of_before_take_the_workspace_they_took():
    """The block's column sums make the size function's answer larger; the other calls need what they needed."""
    D = moe.make_dims(**dict(BASE, T=4096, d=4096))
    from test_train_cpu import _calls as before
    need = 256 + 128 * 2 * 8 * 4  # the error word, the router gradient's partial sums
    for call in ("gate_grad", "up", "down", "down_grad"):
        assert before(D, n=need - 1)[call]() == moe.MOE_ERR_CAPACITY
    # with enough of it a call goes on to the next check
    assert before(D, n=need, bal=-1.0)["gate_grad"]() == moe.MOE_ERR_INVALID_ARG
    assert before(D, n=need, null="h")["down"]() == moe.MOE_ERR_INVALID_ARG


# ---------------------------------------------------------------- the binding, on a machine whose current device is 0

def _device_calls(dev):
    import torch
    from test_train_device_cpu import I, I32, F32, M, N, T, d, on

    def t(name, *shape, dtype=torch.bfloat16):
        return name, on(dev(name), *shape, dtype=dtype)

    def packed(name, rows, cols):
        nb = (cols + 31) // 32
        return [t(name + "_q", rows, nb * 32, dtype=torch.int8), t(name + "_scale", rows, nb, dtype=torch.uint8)]

    ws, off = t("ws", 64, dtype=torch.uint8), t("expert_offsets", N + 1, dtype=I32)
    tok = lambda n: t(n, T, dtype=F32)  # noqa: E731
    col = lambda n, dt=torch.bfloat16: t(n, d, dtype=dt)  # noqa: E731
    D, B = moe.make_dims(T, d, N, 2, I), moe.make_block(gate=moe.MOE_GATE_TOKEN)
    w = lambda n: t(n, N, I, d)  # noqa: E731
    return {
        "moe_norm_rows": [D, t("x", T, d), col("weight"), 1e-6, 0.0, t("n", T, d), tok("rstd")],
        "moe_norm_rows_grad": [D, t("dn", T, d), t("x", T, d), tok("rstd"), col("weight"), 0.0, t("add", T, d), t("dx", T, d),
                               col("dweight", F32), True, ws],
        "moe_block_out": [D, B, t("y", T, d), t("residual", T, d), tok("gate"), col("w_post"), col("w_next"), t("out", T, d),
                          t("next", T, d), tok("rstd_post"), tok("rstd_next")],
        "moe_block_out_grad": [D, B, t("dout", T, d), t("dnext", T, d), t("y", T, d), t("out", T, d), tok("gate"), col("w_post"),
                               col("w_next"), tok("rstd_post"), tok("rstd_next"), t("dresidual", T, d), t("dy", T, d), tok("dgate"),
                               col("dw_post"), col("dw_next"), False, ws],
        "moe_pack_rows": [t("x", T, d), *packed("x", T, d)],
        "moe_unpack_rows": [*packed("x", T, d), t("index", M, dtype=I32), 2, t("out", M, d)],
        "moe_experts_up_packed": [D, t("x_perm", M, d), off, w("w_gate"), w("w_up"), *packed("g", M, I), *packed("u", M, I),
                                  t("h", M, I), ws],
        "moe_experts_down_grad_packed": [D, t("dy_perm", M, d), *packed("g", M, I), *packed("u", M, I), off, w("w_down"), t("h", M, I),
                                         t("dg", M, I), t("du", M, I), w("dw_down"), False, ws],
        "moe_combine_rows_grad_packed": [D, t("dout", T, d), *packed("y", M, d), t("gate", M, dtype=F32), t("inv_perm", M, dtype=I32),
                                         t("dy_perm", M, d), t("dgate", M, dtype=F32)],
    }


@pytest.fixture
def queued(monkeypatch):
    import torch

    from expert_routing_ffn_gb300 import train
    made = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or moe.MOE_OK

    monkeypatch.setattr(train, "lib", Lib)
    monkeypatch.setattr(train, "_here", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0)
    return made


NAMES = [(c, a[0]) for c, args in _device_calls(lambda n: 0).items() for a in args if isinstance(a, tuple)]


def _run(call, dev):
    getattr(moe, call)(*(a[1] if isinstance(a, tuple) else a for a in _device_calls(dev)[call]))


@pytest.mark.parametrize("call", sorted({c for c, _ in NAMES}))
def test_tensors_of_the_current_device_are_taken(call, queued):
    _run(call, lambda n: 0)
    assert queued == [call]


@pytest.mark.parametrize("call,name", NAMES)
def test_a_tensor_of_another_device_is_refused(call, name, queued):
    with pytest.raises(ValueError, match=f"{name} is on cuda:1"):
        _run(call, lambda n: 1 if n == name else 0)
    assert not queued


def test_binding_refuses_wrong_types_and_shapes(queued):
    import torch
    from test_train_device_cpu import on
    args = [a[1] if isinstance(a, tuple) else a for a in _device_calls(lambda n: 0)["moe_block_out"]]
    with pytest.raises(TypeError, match="y has dtype"):
        moe.moe_block_out(*args[:2], on(0, 4, 40, dtype=torch.float16), *args[3:])
    with pytest.raises(ValueError, match="no gate"):
        moe.moe_block_out(args[0], moe.make_block(), *args[2:])
    with pytest.raises(TypeError, match="dtype"):
        moe.moe_pack_rows(on(0, 4, 40, dtype=torch.float16), on(0, 4, 64, dtype=torch.int8), on(0, 4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError, match="scale must be"):
        moe.moe_unpack_rows(on(0, 4, 64, dtype=torch.int8), on(0, 4, 2, dtype=torch.uint8), None, 1, on(0, 4, 65))
    grad = [a[1] if isinstance(a, tuple) else a for a in _device_calls(lambda n: 0)["moe_block_out_grad"]]
    with pytest.raises(TypeError, match="dw_next"):  # the sums over the tokens share a type
        moe.moe_block_out_grad(*grad[:15], on(0, 40, dtype=torch.float32), *grad[16:])
    assert not queued
