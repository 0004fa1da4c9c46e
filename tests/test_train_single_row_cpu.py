"""Token rows of a wider tensor in the binding: rows keep their stride, a single
row is d values whatever stands behind it."""
import pytest
import torch

import expert_routing_ffn_gb300.train as train

HERE = -1  # a CPU tensor's device, as the binding sees it


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_single_row_has_the_stride_of_its_columns(dtype):
    wide = torch.zeros((4, 2049), dtype=dtype)
    for rows, T, ld in ((wide[:, :2048], 4, 2049), (wide[1:3, :2048], 2, 2049), (wide[2:3, :2048], 1, 2048), (wide[:, :2048], 1, 2048)):
        assert train._rows(HERE, rows, dtype, T, 2048, "x") == (rows.data_ptr(), ld)
    assert train._plain_rows(HERE, wide[:, :2048], "x")[1:4] == (2048, wide.data_ptr(), 2049)
    assert train._plain_rows(HERE, wide[1:2, :2048], "x")[:4] == (1, 2048, wide[1:2].data_ptr(), 2048)


def test_rows_that_overlap_or_lie_apart_are_still_refused():
    t = torch.zeros((4, 8))
    for bad in (t[:, ::2], t.expand(4, 8)[0:1].expand(4, 8), t.t()):
        with pytest.raises(ValueError):
            train._rows(HERE, bad, torch.float32, bad.shape[0], bad.shape[1], "x")
