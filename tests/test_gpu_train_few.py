"""The experts' products on the CUDA cores with few rows an expert: on both
sides of the row counts where the kernels change, rows longer than a block
holds at a time, ragged columns, and sizes without 16-byte loads."""
import pytest

from test_gpu_train_large import test_every_product_at_the_edges as every_product

pytestmark = pytest.mark.gpu

CASES = [  # T, d, N, k, I, routing, type
    (12, 1100, 8, 2, 700, "some", "f32"), (12, 1101, 8, 2, 699, "some", "f32"), (12, 1101, 8, 2, 699, "some", "bf16"),
    (24, 520, 8, 2, 516, "all", "f32"), (25, 520, 8, 2, 516, "all", "f32"), (64, 132, 8, 2, 68, "all", "f32"),
    (65, 132, 8, 2, 68, "all", "f32"), (96, 36, 4, 1, 100, "one", "f32"), (100, 513, 10, 2, 35, "skew", "bf16"),
    (97, 33, 2, 2, 65, "all", "bf16"), (96, 33, 2, 2, 65, "all", "bf16"), (1, 1025, 3, 1, 1, "all", "f32"),
    (8, 4, 16, 4, 4, "all", "f32"), (9, 2, 2, 1, 3, "one", "bf16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_products_of_few_rows(case):
    every_product(case)
