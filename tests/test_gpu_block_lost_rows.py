"""Norms of long batches whose wait for a row runs out: the calls end, the row
and those that its group of threads still had become NaN, all others keep their
values, the gradients report it, and the calls after them are what they were."""
import numpy as np
import pytest
import torch

import expert_routing_ffn_gb300 as moe
from test_gpu_block import dims, vec
from test_gpu_train import clean, empty, rnd, workspace

pytestmark = pytest.mark.gpu

# d, type, rows an SM works on at a time at most: groups of one warp, of several, one of the largest (where a norm
# alone does not go through shared memory)
SHAPES = [(264, "f32", 12), (1536, "bf16", 8), (8192, "bf16", 1)]
CASES = [(call, *s) for call in ("norm", "norm_grad", "block", "block_grad") for s in SHAPES if not (call == "norm" and s[0] == 8192)]


@pytest.fixture
def lose():
    yield moe.moe_testing_lose_row
    moe.moe_testing_lose_row(-1)


def _same_but_lost(got, good, row, sms):
    """The rows that are NaN: row and every G-th after it, G a multiple of the SMs; the others bit for bit."""
    lost = got.isnan().reshape(got.shape[0], -1)
    assert torch.equal(lost.any(1), lost.all(1))
    rows = torch.nonzero(lost[:, 0]).flatten().tolist()
    assert rows and rows[0] == row
    if len(rows) > 1:
        G = rows[1] - row
        assert G % sms == 0 and rows == list(range(row, got.shape[0], G))
    keep = ~lost[:, 0]
    assert torch.equal(got[keep], good[keep])
    return rows


@pytest.mark.parametrize("call,d,kind,most", CASES)
def test_a_row_that_never_arrives(call, d, kind, most, lose):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 4 * sms * most + 3
    rng = np.random.default_rng(T)
    D, B = dims(T, d, kind), moe.make_block(gate=moe.MOE_GATE_TOKEN)
    x, y, z = (rnd(rng, (T, d), kind)[0] for _ in range(3))
    w = vec(rng, d, kind, 0.2, 1.0)[0]
    r, gate = vec(rng, T, "f32", 0.1, 1.0)[0], vec(rng, T, "f32", 0.1, 1.0)[0]
    ws = workspace(D)

    def run():
        rows, sums = [empty((T, d), kind)], []
        if call == "norm":
            rows.append(empty((T,), "f32"))
            moe.moe_norm_rows(D, x, w, 1e-6, 0.0, *rows)
        elif call == "norm_grad":
            sums = [empty((d,), "f32")]
            moe.moe_norm_rows_grad(D, x, y, r, w, 0.0, None, rows[0], sums[0], False, ws)
        elif call == "block":
            rows += [empty((T, d), kind), empty((T,), "f32"), empty((T,), "f32")]
            moe.moe_block_out(D, B, y, x, gate, w, w, *rows)
        else:
            rows += [empty((T, d), kind), empty((T,), "f32")]
            sums = [empty((d,), "f32"), empty((d,), "f32")]
            moe.moe_block_out_grad(D, B, x, z, y, x, gate, w, w, r, r, *rows, *sums, False, ws)
        return rows, sums

    good, good_sums = run()
    clean(ws)
    assert not any(bool(t.isnan().any()) for t in good + good_sums)
    row = 3 * sms + 1  # its group's second row or a later one, or its first, by the shape
    lose(row)
    got, sums = run()
    torch.cuda.synchronize()
    lose(-1)
    lost = [_same_but_lost(a, b, row, sms) for a, b in zip(got, good)]
    assert all(v == lost[0] for v in lost)
    assert all(bool(t.isnan().all()) for t in sums)
    st, det = moe.moe_check(ws)
    if call.endswith("grad"):
        G = lost[0][1] - row if len(lost[0]) > 1 else None
        assert st == moe.MOE_ERR_TIMEOUT and det <= row and (G is None or det == row % G)
        clean(ws)
    else:
        assert st == moe.MOE_OK
    again, again_sums = run()
    clean(ws)
    assert all(torch.equal(a, b) for a, b in zip(again + again_sums, good + good_sums))
