"""What the training example's layer holds on the device with activations in 8
bits, and without."""
import os
import sys

import pytest
import torch

from workloads import CONFIGS

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layer,T", [("granite", 512), ("dsv2lite", 256)])
def test_packed_activations_take_less_than_those_in_16_bits(layer, T):
    from train_step import TrainLayer
    cfg = CONFIGS[layer]

    def held(packed):
        L = TrainLayer(cfg, T, packed=packed)
        tensors = [t for v in vars(L).values() for t in (v if isinstance(v, tuple) else (v,)) if isinstance(t, torch.Tensor)]
        return sum({t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in tensors}.values())

    # a slot: g, u and a row of dx in 16 bits less; g, u, y (and a k-th of x) in 8 bits with their scales more
    d, I, k = cfg.d, cfg.I, cfg.k
    nb = lambda c: (c + 31) // 32 * 33  # noqa: E731
    less = T * k * (2 * (2 * I + d) - 2 * nb(I) - nb(d)) - T * nb(d)
    assert less > 0 and held(False) - held(True) == less
