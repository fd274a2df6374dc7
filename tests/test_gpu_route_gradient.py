"""The router's gradient on what callers may hand back to it, against the fp64
definition in oracle.rows.

Tolerance, as derived for the router's other tests: 400 u of the sum of the
terms' magnitudes (u = 2^-24), and half a step of the result's type."""
import numpy as np
import pytest
import torch

from oracle import rows as ref
from tests.test_gpu_rows import HALF_BF16, U, near, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


def logits_of(T, E, dtype, seed):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).mul(2).to(dtype)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_weights", [True, False])
@pytest.mark.parametrize("E", [5, 16, 64, 100, 256, 1024])
def test_ids_outside_the_experts_are_none(fp8, E, with_weights, renorm, scoring):
    """An id below 0 or from E on counts as -1, wherever in the row it stands; a
    row with no other ids chose nothing and gets zeros, from the loss too."""
    T, k = 40, 4
    z = logits_of(T, E, torch.float32, E)
    zd = z.cuda()
    ids, _, _, _, slope = fp8.route(zd, k, scoring, renorm, 2.0, 0.5)
    ids[0] = E
    ids[1] = torch.tensor([E, E + 1, 2 ** 31 - 1, -1])
    ids[2] = torch.tensor([-1, -7, -2 ** 31, E])
    ids[3, 0] = E
    ids[4, :3] = -5
    ids[5, 1] = 2 ** 31 - 1
    ids[6] = -1
    dw = torch.from_numpy(np.random.default_rng(E).standard_normal((T, k)).astype(np.float32)).cuda() \
        if with_weights else None
    d = fp8.route_backward(zd, ids, dw, slope, None, scoring, renorm, 2.0)
    fp8.check()
    assert (d[[0, 1, 2, 6]] == 0).all()
    want = ref.route_backward(np64(z), ids.cpu().numpy(), None if dw is None else np64(dw), np64(slope), 1.0, scoring,
                              renorm, 2.0)
    mag = 2 * np.abs(np64(slope)).max() + (0 if dw is None else 8 * np.abs(np64(dw)).max())
    near(np64(d), want, 400 * U * mag, "d_logits")
