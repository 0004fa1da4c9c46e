"""The combine's gradient from packed rows where a product of dout with a whole
number of steps would pass float32's range, though dout y does not, and where
it would fall below it."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
import train_ref
from test_gpu_packed import given
from test_gpu_train import TYPES, dev, empty, host, routing
from train_ref import STEP, check, rounded

pytestmark = pytest.mark.gpu


# dout's and y's size: dout up to the type's largest value (a step of y is 2^-20 and less), eight products of one sign
# included; dout near the smallest normal value beside large steps; y below the normal values (steps of 2^-127)
@pytest.mark.parametrize("dsize,ysize", [(1e38, 1e-4), (3e38, 1e-30), (1e-37, 1e36), (1e30, 1e-37)])
@pytest.mark.parametrize("T,d,k,kind", [(33, 264, 8, "bf16"), (33, 264, 16, "f32"), (5, 251, 3, "f32"), (7, 12000, 2, "bf16")])
def test_products_of_dout_and_y_keep_their_range(T, d, k, kind, dsize, ysize):
    rng = np.random.default_rng(T + d)
    N = 32
    D = moe.make_dims(T, d, N, k, 64, wtype=kind)
    _, _, inv = train_ref.sort_slots(routing(rng, T, N, k, "some"), N, 0)
    sign = np.where(rng.random((T, d)) < 0.5, -1.0, 1.0)
    sign[0] = 1.0
    t = torch.from_numpy((sign * rng.uniform(0.5, 1.0, (T, d)) * dsize).astype(np.float32)).to(TYPES[kind])
    dout, doh = t.cuda(), t.double().numpy()
    assert np.isfinite(doh).all()
    y = rng.standard_normal((T * k, d))
    y[:2] = np.abs(y[:2])
    rq, rE = ref.pack((y * ysize).astype(np.float32).astype(np.float64))
    y = ref.unpack(rq, rE, d)
    q, e = given(rq, rE)
    dy, dgate = empty((T * k, d), kind), empty((T, k), "f32")
    moe.moe_combine_rows_grad_packed(D, dout, q, e, None, dev(inv), dy, dgate)
    edy, edg, mag = train_ref.combine_grad(doh, y, None, inv)
    assert np.max(mag) < 1e38  # every sum of some of the terms is in range
    check(host(dy), edy, rounded(edy, 4 * STEP * np.abs(edy), kind), "dy")
    check(host(dgate), edg, train_ref.bound(edg, d, mag, "f32"), "dgate")
