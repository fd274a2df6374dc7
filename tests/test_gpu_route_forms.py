"""The router's three forms (one block, one cluster, the grid) on both sides of
their borders, against the fp64 definition in oracle.rows."""
import numpy as np
import pytest
import torch

from tests.test_gpu_rows import check_route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,rows", [(16, 128), (64, 128), (100, 64), (256, 32), (512, 16), (1024, 8)])
def test_on_both_sides_of_the_borders(fp8, E, rows, scoring):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for T in (rows - 1, rows, rows + 1, 8 * rows - 1, 8 * rows, 8 * rows + 1, 9 * rows + 3,
              *((sms * rows, sms * rows + 1) if rows <= 16 else ())):
        z = torch.randn(T, E, generator=torch.Generator().manual_seed(T)) * 2
        mask = np.random.default_rng(T).random(T) < 0.9
        check_route(fp8, z, 4, scoring, True, mask=mask, label=f"{T} x {E}")
