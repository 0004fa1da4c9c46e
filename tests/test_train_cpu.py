"""The training step without a GPU: the gradients' formulas against central
differences of the forward formulas (64 bits), the calls' refusals, and the
workspace's size."""
import ctypes as C

import numpy as np
import pytest

import expert_routing_ffn_gb300 as moe
import train_ref as ref


def _slope(f, x, v, eps=1e-5):
    """Central difference of f along v."""
    return (f(x + eps * v) - f(x - eps * v)) / (2 * eps)


def _case(seed=0, T=5, d=6, N=4, k=2, I=3, drop=True):
    rng = np.random.default_rng(seed)
    logits = rng.normal(size=(T, N))
    prob = np.exp(logits) / np.exp(logits).sum(1, keepdims=True)
    idx = np.argsort(-prob, 1)[:, :k].astype(np.int32)
    if drop:
        idx[1, 0] = -1
        idx[3, :] = -1
    off, perm, inv = ref.sort_slots(idx, N, 0)
    w = [rng.normal(size=(N, I, d)) * 0.5 for _ in range(3)]
    return rng, logits, prob, idx, off, perm, inv, w


# central differences at eps = 1e-5 of smooth functions of order 1 in float64:
# truncation ~ eps^2 = 1e-10, cancellation ~ 1e-16 / eps = 1e-11 of the loss
DIFF_TOL = 1e-7


@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_formula_matches_differences(renorm):
    rng, logits, _, idx, *_ = _case()
    dgate = rng.normal(size=idx.shape)
    c = 0.3
    load = ref.load_of(idx, logits.shape[1])

    def loss(l):
        p = np.exp(l) / np.exp(l).sum(1, keepdims=True)
        return float((dgate * ref.gates(p, idx, renorm))[idx >= 0].sum()) + ref.balance_loss(p, load, c)

    prob = np.exp(logits) / np.exp(logits).sum(1, keepdims=True)
    dl, _, _ = ref.gate_grad(prob, idx, dgate, renorm, c)
    for _ in range(4):
        v = rng.normal(size=logits.shape)
        assert abs(_slope(loss, logits, v) - float((dl * v).sum())) <= DIFF_TOL


def test_whole_chain_of_formulas_matches_differences():
    """dispatch -> up -> down -> combine: the chain of the gradient formulas
    is the derivative of the chain of the forward formulas, for x, the gates
    and the three weights."""
    rng, _, prob, idx, off, perm, inv, (wg, wu, wd) = _case(1)
    k = idx.shape[1]
    x, add = rng.normal(size=(idx.shape[0], wg.shape[2])), rng.normal(size=(idx.shape[0], wg.shape[2]))
    gate, r = ref.gates(prob, idx, False), rng.normal(size=x.shape)

    def forward(x, gate, wg, wu, wd):
        xp = ref.dispatch(x, perm, k)
        h = ref.experts_up(xp, off, wg, wu)[2]
        y = ref.experts_down(h, off, wd)[0]
        return float((r * ref.combine(y, gate, inv, add)[0]).sum())

    xp = ref.dispatch(x, perm, k)
    g, u, h, _, _ = ref.experts_up(xp, off, wg, wu)
    y = ref.experts_down(h, off, wd)[0]
    dy, dgate, _ = ref.combine_grad(r, y, gate, inv)
    dg, du, _, _ = ref.experts_dh(dy, g, u, off, wd)
    grads = [ref.combine(ref.experts_dx(dg, du, off, wg, wu)[0], None, inv, None)[0], dgate,
             ref.experts_dw(dg, xp, off, wg.shape[0])[0], ref.experts_dw(du, xp, off, wg.shape[0])[0],
             ref.experts_dw(h, dy, off, wg.shape[0])[0]]
    at = [x, gate, wg, wu, wd]
    for i, grad in enumerate(grads):
        v = rng.normal(size=at[i].shape)
        f = lambda z: forward(*[z if j == i else at[j] for j in range(5)])  # noqa: E731
        assert abs(_slope(f, at[i], v) - float((grad * v).sum())) <= DIFF_TOL * max(1.0, abs(float((grad * v).sum())))


BASE = dict(T=4, d=40, N=8, k=2, I=24, wtype="bf16")


@pytest.mark.parametrize("kw,status", [
    (dict(N=513), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=17, N=32), moe.MOE_ERR_UNSUPPORTED),
    (dict(k=9, N=8), moe.MOE_ERR_UNSUPPORTED),
    (dict(T=1 << 24, k=2), moe.MOE_ERR_UNSUPPORTED),
    (dict(d=1 << 17), moe.MOE_ERR_UNSUPPORTED),
    (dict(I=1 << 17), moe.MOE_ERR_UNSUPPORTED),
    (dict(T=-1), moe.MOE_ERR_INVALID_ARG),
    (dict(d=0), moe.MOE_ERR_INVALID_ARG),
    (dict(I=0), moe.MOE_ERR_INVALID_ARG),
    (dict(k=0), moe.MOE_ERR_INVALID_ARG),
])
def test_bad_dims_are_refused_by_every_call(kw, status):
    D = moe.make_dims(**dict(BASE, **kw))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_train_workspace_size(D)
    assert e.value.status == status
    assert moe.moe_experts_path(D) == "unsupported"
    for call in _calls(D).values():
        assert call() == status


@pytest.mark.parametrize("dims", [BASE, dict(BASE, T=0), dict(BASE, N=512, k=16, T=1 << 20), dict(BASE, T=1 << 23)])
def test_workspace_stays_below_its_documented_limit(dims):
    assert 0 < moe.moe_train_workspace_size(moe.make_dims(**dims)) <= 16 << 20


A, B, F, WS = 0x10000, 0x20000, 0x30000, 1 << 20  # addresses that a refused call never follows


def _calls(D, null=None, ws=WS, n=16 << 20, ld=0, cap=0, g=moe.MOE_DTYPE_BF16, acc=0, bal=0.0, odd=None):
    """Every call with made-up addresses; argument `null` is NULL, `odd` misaligned."""
    L, r = moe.lib(), C.byref(D)

    def a(name, v=A):
        return None if null == name else v + 1 if odd == name else v

    return {
        "dispatch": lambda: L.moe_dispatch_rows(r, a("x"), ld, a("idx"), cap, a("x_perm"), a("off"), a("perm"),
                                                a("inv"), ws, n, None),
        "dispatch_grad": lambda: L.moe_dispatch_rows_grad(r, a("y"), a("inv"), a("add"), ld, a("out"), ld, None),
        "combine": lambda: L.moe_combine_rows(r, a("y"), a("gate"), a("inv"), a("add"), ld, a("out"), ld, None),
        "combine_grad": lambda: L.moe_combine_rows_grad(r, a("dout"), ld, a("y"), a("gate"), a("inv"), a("dy"),
                                                        a("dgate"), None),
        "gate_grad": lambda: L.moe_gate_grad(r, a("prob"), a("idx"), a("dgate"), bal, a("dlogits"), a("loss"), ws, n,
                                             None),
        "up": lambda: L.moe_experts_up(r, a("x_perm"), a("off"), a("wg"), a("wu"), a("g"), a("u"), a("h"), ws, n, None),
        "up_grad": lambda: L.moe_experts_up_grad(r, a("dg"), a("du"), a("x_perm"), a("off"), a("wg"), a("wu"),
                                                 a("dx"), a("dwg"), a("dwu"), g, acc, ws, n, None),
        "down": lambda: L.moe_experts_down(r, a("h"), a("off"), a("wd"), a("y"), ws, n, None),
        "down_grad": lambda: L.moe_experts_down_grad(r, a("dy"), a("h"), a("g"), a("u"), a("off"), a("wd"), a("dg"),
                                                     a("du"), a("dwd"), g, acc, ws, n, None),
    }


REQUIRED = [("dispatch", n) for n in ("x", "idx", "x_perm", "off", "perm", "inv")] + \
    [("dispatch_grad", n) for n in ("y", "inv", "out")] + [("combine", n) for n in ("y", "inv", "out")] + \
    [("combine_grad", n) for n in ("dout", "inv", "y")] + \
    [("gate_grad", n) for n in ("prob", "idx", "dgate", "dlogits")] + \
    [("up", n) for n in ("x_perm", "off", "wg", "wu", "h", "g", "u")] + \
    [("up_grad", n) for n in ("dg", "du", "x_perm", "off", "wg", "wu", "dwg", "dwu")] + \
    [("down", n) for n in ("h", "off", "wd", "y")] + \
    [("down_grad", n) for n in ("dy", "h", "g", "u", "off", "wd", "dg", "du")]


@pytest.mark.parametrize("call,arg", REQUIRED)
def test_missing_buffers_are_refused_before_cuda(call, arg):
    assert _calls(moe.make_dims(**BASE), null=arg)[call]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call,arg", [("dispatch", "x"), ("combine", "add"), ("combine_grad", "dy"), ("up", "wg"),
                                      ("up_grad", "dwu"), ("down", "y"), ("down_grad", "dwd")])
def test_rows_off_an_element_boundary_are_refused(call, arg):
    assert _calls(moe.make_dims(**BASE), odd=arg)[call]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("call,arg", [("dispatch", "idx"), ("dispatch", "off"), ("dispatch", "perm"), ("dispatch", "inv"),
                                      ("combine", "gate"), ("combine", "inv"), ("combine_grad", "gate"),
                                      ("combine_grad", "dgate"), ("gate_grad", "prob"), ("gate_grad", "dlogits"),
                                      ("gate_grad", "loss"), ("up", "off"), ("up_grad", "off"), ("down", "off"),
                                      ("down_grad", "off")])
def test_indices_and_floats_off_a_word_boundary_are_refused(call, arg):
    assert _calls(moe.make_dims(**BASE), odd=arg)[call]() == moe.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,path", [
    (dict(), "simt"), (dict(d=64, I=64), "tc"), (dict(d=2048, I=1408), "tc"), (dict(d=72, I=200), "tc"),
    (dict(d=100, I=64), "simt"), (dict(d=64, I=60), "simt"), (dict(d=56, I=64), "simt"), (dict(d=64, I=56), "simt"),
    (dict(d=2048, I=1408, wtype="f32"), "simt"), (dict(N=512, d=64, I=64), "tc"),
])
def test_products_path_choice(kw, path):
    assert moe.moe_experts_path(moe.make_dims(**dict(BASE, **kw))) == path


def test_workspace_stride_capacity_and_type_refusals():
    D = moe.make_dims(**BASE)
    for call in ("dispatch", "gate_grad", "up", "up_grad", "down", "down_grad"):
        assert _calls(D, ws=None)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, ws=WS + 8)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, n=moe.moe_train_workspace_size(D) - 1)[call]() == moe.MOE_ERR_CAPACITY
    for call in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
        assert _calls(D, ld=39)[call]() == moe.MOE_ERR_INVALID_ARG
        assert _calls(D, ld=-64)[call]() == moe.MOE_ERR_INVALID_ARG
    assert _calls(D, cap=-1)["dispatch"]() == moe.MOE_ERR_INVALID_ARG
    for bal in (-0.5, float("nan"), float("inf")):
        assert _calls(D, bal=bal)["gate_grad"]() == moe.MOE_ERR_INVALID_ARG
    for call in ("up_grad", "down_grad"):
        assert _calls(D, acc=1)[call]() == moe.MOE_ERR_UNSUPPORTED         # accumulation into bf16
        assert _calls(D, g=7)[call]() == moe.MOE_ERR_UNSUPPORTED
    F32 = moe.make_dims(**dict(BASE, wtype="f32"))
    for call in ("up_grad", "down_grad"):
        assert _calls(F32, g=moe.MOE_DTYPE_BF16)[call]() == moe.MOE_ERR_UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    D = moe.make_dims(**BASE)
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        moe.moe_dispatch_rows_grad(D, x, x, None, x)
    with pytest.raises(ValueError):
        moe.moe_combine_rows(D, x, None, x, None, None)
