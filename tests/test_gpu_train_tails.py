"""SwiGLU far out on either side: pre-activations at which the sigmoid is as
small as float32 can hold, where h, dg and du are still numbers of the layer's
type.

With s the kernel's sigmoid of an exact g, |s - exact| <= E s + 2^-149: the
second term is float32's spacing below 2^-126; E is 18 steps of 2^-23 where the
exponential is within 2 (float32 layers and the CUDA cores), and the fast
exponential's documented 2 + 1.173 |g| steps more on the tensor cores."""
import numpy as np
import pytest

import expert_routing_ffn_gb300 as moe
import train_ref as ref
from test_gpu_train import clean, dev, empty, host, rnd, workspace

pytestmark = pytest.mark.gpu

# exact in bf16; e^-g passes 2^126 at 87.34 and float32's largest value at 88.72, and s falls below 2^-149 at 103.3
TAILS = np.array([-20, -60, -80, -86.5, -87.5, -88, -88.5, -89, -92, -96, -100, 0, 20, 60, 80, 87.5, 88.5, 100, -1.5, 3])

CASES = [  # T, d, N, k, I, type: which kernels
    (16, 64, 4, 2, 64, "bf16"), (300, 72, 3, 2, 136, "bf16"),                       # tensor cores, 64-row and 256-row tiles
    (16, 37, 4, 2, 29, "bf16"), (300, 37, 2, 1, 29, "bf16"),                        # CUDA cores, few rows and many
    (8, 64, 4, 2, 64, "f32"), (40, 64, 4, 1, 64, "f32"), (300, 64, 3, 2, 40, "f32"),  # the same in float32, and 16-row tiles
]


def setting(T, N, k, rng):
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32)
    off, _, _ = ref.sort_slots(idx, N, 0)
    return off, dev(off)


def sigmoid_error(g, s, fast):
    return s * (18 + (2 + 1.173 * np.abs(g) if fast else 0)) * ref.STEP + 2.0 ** -149


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_up_in_the_tails(case):
    T, d, N, k, I, kind = case
    rng = np.random.default_rng(T + d)
    D = moe.make_dims(T, d, N, k, I, wtype=kind)
    off, doff = setting(T, N, k, rng)
    # rows that pick one column of the weights: g and u are those values, exactly
    x, _ = rnd(rng, (T * k, d), kind, 0.0)
    x[:, 3] = 1.0
    wg, _ = rnd(rng, (N, I, d), kind)
    wu, _ = rnd(rng, (N, I, d), kind, 2.0 ** 30)
    wg[:, :, 3] = dev(np.resize(TAILS, (N, I))).to(wg.dtype)
    gw, uw = host(wg[:, :, 3]), host(wu[:, :, 3])
    g, u, h = (empty((T * k, I), kind) for _ in range(3))
    ws = workspace(D)
    moe.moe_experts_up(D, x, doff, wg, wu, g, u, h, ws)
    clean(ws)
    expert = np.repeat(np.arange(N), np.diff(off))
    eg, eu = gw[expert], uw[expert]
    assert np.array_equal(host(g), eg) and np.array_equal(host(u), eu)
    s = ref.sigmoid(eg)
    eh = eg * s * eu
    off_h = np.abs(eg * eu) * sigmoid_error(eg, s, moe.moe_experts_path(D) == "tc") + 4 * ref.STEP * np.abs(eh) + 2.0 ** -149 * np.abs(eu)
    ref.check(host(h), eh, ref.rounded(eh, off_h, kind), "h")


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_down_gradient_in_the_tails(case):
    T, d, N, k, I, kind = case
    rng = np.random.default_rng(T + I)
    D = moe.make_dims(T, d, N, k, I, wtype=kind)
    off, doff = setting(T, N, k, rng)
    dy, dyh = rnd(rng, (T * k, d), kind)
    wd, wdh = rnd(rng, (N, I, d), kind, 2.0 ** 15)
    u, uh = rnd(rng, (T * k, I), kind, 2.0 ** 15)
    gh = np.resize(TAILS, (T * k, I))
    g = dev(gh).to(u.dtype)
    dg, du = empty((T * k, I), kind), empty((T * k, I), kind)
    ws = workspace(D)
    moe.moe_experts_down_grad(D, dy, None, g, u, doff, wd, dg, du, None, False, ws)
    clean(ws)
    edg, edu, og, ou = ref.experts_dh(dyh, gh, uh, off, wdh)
    # beside experts_dh's terms, the sigmoid's: d(dg)/ds <= |dh u| (1 + |g|), d(du)/ds = dh g
    dh = np.zeros((T * k, I))
    for e, r in ref.by_expert(off):
        dh[r] = np.abs(dyh[r]) @ np.abs(wdh[e]).T
    ds = sigmoid_error(gh, ref.sigmoid(gh), moe.moe_experts_path(D) == "tc")
    og, ou = og + dh * np.abs(uh) * (1 + np.abs(gh)) * ds, ou + dh * np.abs(gh) * ds
    ref.check(host(dg), edg, ref.rounded(edg, og, kind), "dg")
    ref.check(host(du), edu, ref.rounded(edu, ou, kind), "du")
