"""The router's gradient where a token's gates are renormalised over a small
sum: the probabilities of its live slots add up to as little as float32's
smallest value, and the gradient stays the finite one of the formula."""
import numpy as np
import pytest
import torch

import expert_routing_ffn_gb300 as moe
import train_ref as ref
from test_gpu_train import clean, dev, empty, host, workspace

pytestmark = pytest.mark.gpu

# the live slots' sum, token by token: ordinary, at the smallest normal value 2^-126 = 1.2e-38 and on either side of
# it, below 2^-128 = 2.9e-39 (whose reciprocal is no float32 number), and down to the smallest subnormal 1.4e-45
SUMS = [0.3, 1e-30, 1e-37, 2e-38, 1e-38, 4e-39, 2e-39, 1e-40, 3e-43, 5e-45, 1.5e-45, 0.0]


@pytest.mark.parametrize("N,k", [(8, 3), (40, 8), (300, 16)])
@pytest.mark.parametrize("balance", [0.0, 0.5])
@pytest.mark.parametrize("size", [1.0, 1e4])
def test_gates_renormalised_over_a_small_sum(N, k, balance, size):
    rng = np.random.default_rng(N)
    T = len(SUMS)
    D = moe.make_dims(T, 16, N, k, 8, wtype="bf16", renorm_topk=1)
    idx = np.stack([rng.permutation(N)[:k] for _ in range(T)]).astype(np.int32)
    share = rng.random((T, k)) + 0.1
    share[:, 0] = 0.0
    prob = np.zeros((T, N), np.float32)
    np.put_along_axis(prob, idx, (share / share.sum(1, keepdims=True) * np.array(SUMS)[:, None]).astype(np.float32), 1)
    prob[np.arange(T), idx[:, 0]] = 1.0 - prob.sum(1)  # the confident choice, which no expert takes
    idx[:, 0] = -1
    dgate = (rng.standard_normal((T, k)) * size).astype(np.float32)
    ws, dl, loss = workspace(D), empty((T, N), "f32"), empty((1,), "f32")
    moe.moe_gate_grad(D, dev(prob), dev(idx), dev(dgate), balance, dl, loss, ws)
    clean(ws)
    edl, _, mag = ref.gate_grad(prob.astype(np.float64), idx, dgate.astype(np.float64), True, balance)
    ref.check(host(dl), edl, ref.bound(edl, N + 2 * k + 64, mag, "f32"), "dlogits")


def test_one_live_slot_has_no_gradient_through_its_gate():
    """A single live slot's renormalised gate is one whatever its probability."""
    T, N, k = len(SUMS), 8, 2
    D = moe.make_dims(T, 16, N, k, 8, wtype="bf16", renorm_topk=1)
    prob = np.zeros((T, N), np.float32)
    prob[:, 1], prob[:, 5] = 1.0, SUMS
    idx = np.tile(np.array([[-1, 5]], np.int32), (T, 1))
    dgate = np.full((T, k), -7.0, np.float32)
    ws, dl = workspace(D), empty((T, N), "f32")
    moe.moe_gate_grad(D, dev(prob), dev(idx), dev(dgate), 0.0, dl, None, ws)
    clean(ws)
    assert not torch.any(dl)
