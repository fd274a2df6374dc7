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


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_same_bits_beside_any_number_of_closed_experts(fp8, dtype, renorm, scoring):
    """Two open experts and any number of closed ones (-inf): weights and their
    gradient are the same bits, whatever the width that serves the row.  (Sums
    of two terms and zeros do not depend on their order.)"""
    T = 400
    z = logits_of(T, 2, dtype, 3).cuda()
    dw = torch.randn(T, 2, generator=torch.Generator().manual_seed(4)).cuda()
    first = None
    for E in (2, 8, 9, 16, 17, 32, 33, 64, 65, 128, 200, 256, 257, 512, 600, 1024):
        wide = torch.full((T, E), float("-inf"), dtype=dtype, device="cuda")
        wide[:, :2] = z
        ids, w, _, _, _ = fp8.route(wide, 2, scoring, renorm, 2.5)
        d = fp8.route_backward(wide, ids, dw, None, None, scoring, renorm, 2.5)
        assert (d[:, 2:] == 0).all()
        got = ids, w, d[:, :2]
        first = first or got
        for a, b in zip(got, first):
            assert torch.equal(a, b), E


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,k", [(8, 1), (8, 2), (16, 1), (16, 2), (17, 2), (32, 1), (64, 6), (100, 2), (256, 1), (256, 8),
                                 (1000, 8)])
def test_gradient_by_each_rows_own_terms(fp8, E, k, dtype, renorm, scoring):
    """Tolerance from the terms of the row itself.  With A the largest |z - top| and
    |z| of the row a score is off by e = (2.22 A + 8) u; a share, or a part of the
    chosen scores, by two scores, up to 37 additions and a quotient,
    s = 2 e + 40 u; a sum of shares times inputs by s + 37 u + 3 u of the sum of
    magnitudes; 1 - s by e + 3 u.  Together below 3 s + 60 u of
      f_e (q_e (|up_e| + sum q |up|) + r_e (|down_e| + sum r |down|))
    with q the shares, r the scores that carry the weights' gradient (and, where
    these are softmax shares themselves, q_e sum q |down|), f = 1 - s or 1."""
    T, scale = 300, 2.5
    z = logits_of(T, E, dtype, 11 * E + k)
    zd, zz = z.cuda(), np64(z)
    ids, _, _, _, slope = fp8.route(zd, k, scoring, renorm, scale, 0.1)
    i0 = ids.cpu().numpy()
    dw = torch.from_numpy(np.random.default_rng(k).standard_normal((T, k)).astype(np.float32))
    d = fp8.route_backward(zd, ids, dw.cuda(), slope, None, scoring, renorm, scale)
    fp8.check()
    want = ref.route_backward(zz, i0, np64(dw), np64(slope), 1.0, scoring, renorm, scale)
    up, down = np.abs(np64(slope)), scale * np.abs(np64(dw))
    mag = np.zeros((T, E))
    for t in range(T):
        score, share = ref._scores(zz[t], scoring)
        f = np.ones(E) if scoring == "softmax" else 1 - score
        mag[t] = f * share * (up + (share * up).sum())
        r = score[i0[t]] / score[i0[t]].sum() if renorm else score[i0[t]]
        mag[t, i0[t]] += f[i0[t]] * r * (down[t] + (r * down[t]).sum())
        if scoring == "softmax" and not renorm:
            mag[t] += share * (score[i0[t]] * down[t]).sum()
    A = np.maximum(np.abs(zz - zz.max(1, keepdims=True)), np.abs(zz)).max(1, keepdims=True)
    s = (2 * (2.22 * A + 8) + 40) * U
    half = HALF_BF16 if dtype == torch.bfloat16 else U
    near(np64(d), want, (3 * s + 60 * U) * mag + half * np.abs(want) + 1e-38, "d_logits")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [8, 64, 256])
def test_sigmoid_rows_far_below_zero_keep_their_ratios(fp8, E, renorm):
    """Rows whose scores lie on both sides of fp32's range, beside the top one:
    renormalised weights are ratios and stay what they are (e^-40 = 4e-18), with
    their gradient.  |z - top| <= 70: e is off by (2.22 * 70 + 8) u, a ratio by
    twice that and 40 u, below 400 u; a score below 2^-126 may come out as any
    value down to 0."""
    tops = torch.tensor([-19.0, -25.0, -31.0, -40.0, -55.0, -59.5, -61.0, -80.0, -100.0])
    T, k = tops.numel(), 4
    z = torch.full((T, E), -300.0)
    for j, below in enumerate((0.0, 12.5, 40.0, 66.0)):
        z[:, 2 * j + 1] = tops - below
    ids, w, _, _, _ = fp8.route(z.cuda(), k, "sigmoid", renorm, 2.5)
    i0, w0, _, _, _ = ref.route(np64(z), k, "sigmoid", renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), i0)
    near(np64(w), w0, 400 * U * w0 + (0 if renorm else 2.5 * 2.0 ** -126), "weights")
    for j in range(k):
        dw = torch.zeros(T, k)
        dw[:, j] = 1.0
        d = fp8.route_backward(z.cuda(), ids, dw.cuda(), None, None, "sigmoid", renorm, 2.5)
        want = ref.route_backward(np64(z), i0, np64(dw), None, 1.0, "sigmoid", renorm, 2.5)
        r = w0 / 2.5
        mag = np.zeros((T, E))
        np.put_along_axis(mag, i0, 2.5 * r * (np64(dw) + (r * np64(dw)).sum(1, keepdims=True)) if renorm
                          else 2.5 * r * np64(dw), axis=1)
        near(np64(d), want, 2 * 400 * U * mag + 2.5 * 2.0 ** -126, f"d_logits of {j}")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("with_loss", [True, False])
@pytest.mark.parametrize("E", [8, 64, 256])
def test_a_nan_logit_goes_where_the_formula_takes_it(fp8, E, with_loss, renorm, scoring):
    """Beside chosen experts a NaN logit reaches the whole row through the shares;
    without a gradient through them, what the chosen scores' sum reaches, and
    with sigmoid scores on their own nothing."""
    T, k = 12, 3
    z = logits_of(T, E, torch.float32, 5)
    z[2, 1] = float("nan")
    z[7, E - 1] = float("nan")
    zd = z.cuda()
    ids, _, _, _, slope = fp8.route(zd, k, scoring, renorm, 2.0, 0.0)
    dw = torch.from_numpy(np.random.default_rng(E).standard_normal((T, k)).astype(np.float32)).cuda()
    up = torch.full((E,), 0.25, device="cuda") if with_loss else None
    for d_weights in (dw, None):
        d = fp8.route_backward(zd, ids, d_weights, up, None, scoring, renorm, 2.0)
        want = ref.route_backward(np64(z), ids.cpu().numpy(), None if d_weights is None else np64(dw),
                                  None if up is None else np64(up), 1.0, scoring, renorm, 2.0)
        assert np.isnan(want).any() == (with_loss or d_weights is not None and (renorm or scoring == "softmax"))
        near(np64(d), want, 400 * U * (0.5 + 8 * np.abs(np64(dw)).max()), "d_logits")
