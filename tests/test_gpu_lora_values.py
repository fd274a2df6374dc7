"""Values at the ends of the types in the adapters (lora_add), against the fp64
definition."""
import numpy as np
import pytest
import torch

from tests.test_gpu_lora import bounds, make, np64, run

pytestmark = pytest.mark.gpu
# a few rows in one launch, 16-row tiles, 128-row tiles
FORMS = [(1, 8), (9, 16), (40, 8), (64, 64), (40, 128), (300, 128), (1100, 8), (1100, 24), (1100, 64)]


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


@pytest.mark.parametrize("M,R", FORMS)
def test_inner_products_above_the_largest_bf16(fp8, M, R):
    """u between bf16's largest value, 2^128 - 2^120, and fp32's, where the nearest
    bf16 would be an infinity: u is finite, and so is its product with a small
    B.  (u = 2^128 - 2^120 + 2^119 + 2^118, exact in fp32.)"""
    N, K, L = 72, 136, 2
    ids, t = make(M, N, K, R, L, 60, bare=0.0)
    ids[:] = 0
    x, a = torch.zeros(M, K), torch.zeros(L, R, K)
    x[:, 0], x[:, 1], x[:, 2] = (2.0 ** 64 - 2.0 ** 56), 2.0 ** 60, -(2.0 ** 60)
    a[:, :, 0], a[:, :, 1] = 2.0 ** 64, 2.0 ** 59 + 2.0 ** 58
    a[:, 1::2] = -a[:, 1::2]
    t["x"], t["a"] = x.bfloat16(), a.bfloat16()
    t["b"] = (t["b"].float() * 2.0 ** -100).bfloat16()
    t["scales"] = None
    got = run(fp8, t, ids, L)
    want, slack = bounds(t, ids, K, R)
    assert np.isfinite(want).all() and np.abs(want).min() > 0
    assert (np.abs(np64(got) - want) <= slack).all()


@pytest.mark.parametrize("M,R", FORMS)
def test_infinite_inner_products(fp8, M, R):
    """u = +inf or -inf gives +-inf by the sign of B, NaN where two ranks disagree."""
    N, K, L = 64, 64, 1
    ids, t = make(M, N, K, R, L, 61, bare=0.0)
    t["x"][M // 2, 7] = float("inf")
    t["a"][0, :, 7] = 1.0
    t["a"][0, 1, 7] = -1.0
    b = t["b"][0].abs() + 0.125
    b[:, 1] = -b[:, 1]
    b[5, 1] = 0.25                        # +inf and -inf meet in column 5
    t["b"][0] = b
    got = run(fp8, t, ids, L)
    row = got[M // 2].cpu()
    cols = torch.arange(N) != 5
    assert (row[cols] == float("inf")).all() and torch.isnan(row[5])
    keep = torch.arange(M) != M // 2
    assert torch.isfinite(got.cpu()[keep]).all()


def test_an_order_past_the_last_integer(fp8):
    """A full tile whose rows count on past 2^31 - 1: skipped, as all rows outside
    [0, M) are."""
    M, N, K, R = 1100, 64, 64, 8
    ids, t = make(M, N, K, R, 1, 62, bare=0.0)
    d = {k: v.cuda() for k, v in t.items()}
    off, order, _ = fp8.group_rows(torch.zeros(M, dtype=torch.int32, device="cuda"), 1)
    good = fp8.lora_add(d["y"], d["x"], d["a"], d["b"], off, order, scales=d["scales"])
    far = order.clone()
    far[256:384] = torch.from_numpy((2 ** 31 - 64 + np.arange(128)).astype(np.uint32).view(np.int32)).cuda()
    out = torch.full_like(d["y"], 7.0)
    fp8.lora_add(d["y"], d["x"], d["a"], d["b"], off, far, scales=d["scales"], out=out)
    fp8.check()
    keep = torch.ones(M, dtype=torch.bool)
    keep[256:384] = False
    assert torch.equal(out[keep], good[keep]) and (out[256:384] == 7.0).all()
