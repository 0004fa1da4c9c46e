"""Norms whose squares pass float32's range beside an eps that counts there."""
import numpy as np
import pytest
import torch

import block_ref as ref
import expert_routing_ffn_gb300 as moe
from test_gpu_block import dims, vec
from test_gpu_train import TYPES, empty, host
from train_ref import check, rounded

pytestmark = pytest.mark.gpu


def _large(rng, T, d, kind):
    v = np.where(rng.random((T, d)) < 0.5, -1.0, 1.0) * rng.uniform(0.5, 1.0, (T, d)) * 1e19
    t = torch.from_numpy(v.astype(np.float32)).to(TYPES[kind])
    return t.cuda(), t.double().numpy()


# one vector a thread, single values, rows read again, rows through shared memory
@pytest.mark.parametrize("T,d,kind", [(5, 64, "bf16"), (3, 101, "f32"), (2, 9001, "f32"), (3, 8200, "bf16"), (1900, 3584, "bf16"), (1900, 4096, "f32"),
                                      (4, 2, "f32")])
@pytest.mark.parametrize("eps", [3e37, 3.4e38])  # the latter passes the range with a mean that does not
def test_eps_counts_where_the_squares_pass_the_range(T, d, kind, eps):
    rng = np.random.default_rng(d)
    eps = float(np.float32(eps))
    D = dims(T, d, kind)
    (x, xh), (y, yh) = _large(rng, T, d, kind), _large(rng, T, d, kind)
    w, wh = vec(rng, d, kind, 0.2, 1.0)
    n, r = empty((T, d), kind), empty((T,), "f32")
    moe.moe_norm_rows(D, x, w, eps, 0.0, n, r)
    en, on, er, orr = ref.norm(xh, wh, eps, 0.0)
    check(host(r), er, rounded(er, orr, "f32"), "rstd")
    check(host(n), en, rounded(en, on, kind), "n")
    B = moe.make_block(eps, 0.0, 1.0, True)
    out, nxt, ra, rb = empty((T, d), kind), empty((T, d), kind), empty((T,), "f32"), empty((T,), "f32")
    moe.moe_block_out(D, B, y, x, None, w, w, out, nxt, ra, rb)
    f = ref.block(yh, xh, None, "none", wh, wh, eps, 0.0, 1.0, True)
    for name, t, k in (("rstd_post", ra, "f32"), ("rstd_next", rb, "f32"), ("out", out, kind), ("next", nxt, kind)):
        check(host(t), f[name][0], rounded(*f[name], k), name)
