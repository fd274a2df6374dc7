"""GPU parity of the router, the row sort, the weighted sum and their gradients
against the fp64 definitions in oracle.rows.

Tolerances count roundings (u = 2^-24, the fp32 half step; a bf16 result is
rounded once more, half a step 2^-8 of its value):
  weights, shares: expf is within 2 ulp = 4 u, its argument z - m is rounded
    (u |z - m| absolute, so relative in the result), a row's sum adds at most
    32 + 5 rounded terms, and a handful of products and quotients: with
    |z - m| <= 40 that is below (40 + 37 + 23) u each for numerator and sum,
    200 u together.  A sigmoid score below 2^-126 = e^-87.3 is no normal fp32
    number (and none at all below 2^-149): it may come out as any value down
    to 0, so that much is added.
  loss: shares as above, then at most T / (rows in flight) + 32 more additions
    of positive terms: 200 u + (T / 8 + 64) u.
  d_logits: every term is a share or weight (200 u) times differences of
    inputs; 400 u of the sum of the terms' magnitudes.
  weighted sum: k + 1 fused multiply-adds, u each of the magnitudes so far;
    dot products: a lane's chain of H / 128 + 8 and a tree.
"""
import numpy as np
import pytest
import torch

from oracle import rows as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8
INF = float("inf")


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def near(got, want, slack, label):
    got, want, slack = np.asarray(got, np.float64), np.asarray(want, np.float64), np.broadcast_to(slack, np.shape(want))
    assert got.shape == want.shape, label
    assert np.array_equal(np.isnan(got), np.isnan(want)), label + ": NaN in other places"
    ok = ~np.isnan(want)
    bad = ok & ~(np.abs(got - want) <= slack)
    assert not bad.any(), f"{label}: {bad.sum()} of {bad.size} off, worst " \
        f"{np.max((np.abs(got - want) / np.maximum(slack, 1e-300))[ok])} of the tolerance"


def logits_of(T, E, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype)


def check_route(fp8, z, k, scoring, renorm, scale=1.0, balance=0.02, mask=None, seed=0, label=""):
    """Forward and gradient of one set of logits (a CPU tensor)."""
    T, E = z.shape
    zd = z.cuda()
    md = None if mask is None else torch.as_tensor(mask).cuda()
    ids, w, counts, loss, slope = fp8.route(zd, k, scoring, renorm, scale, balance, md)
    fp8.check()
    zz = np64(z)
    i0, w0, c0, l0, s0 = ref.route(zz, k, scoring, renorm, scale, balance, mask)
    assert np.array_equal(ids.cpu().numpy(), i0), label
    assert np.array_equal(counts.cpu().numpy(), c0), label
    near(np64(w), w0, 200 * U * np.abs(w0) + abs(scale) * 2.0 ** -126, label + " weights")
    near(np64(slope), s0, 4 * U * np.abs(s0), label + " slope")
    near(np64(loss)[0], l0, (264 + T / 8) * U * abs(l0), label + " loss")

    g = np.random.default_rng(seed)
    dw = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)).cuda()
    dl = torch.tensor([0.75], device="cuda")
    d = fp8.route_backward(zd, ids, dw, slope, dl, scoring, renorm, scale)
    fp8.check()
    d0 = ref.route_backward(zz, i0, np64(dw), s0, 0.75, scoring, renorm, scale)
    with np.errstate(all="ignore"):
        share = np.array([ref._scores(r, scoring)[1] if np.isfinite(r).any() else np.zeros(E) for r in zz])
    mark = np.zeros((T, E + 1))
    np.put_along_axis(mark, np.where(i0 < 0, E, i0), 1.0, axis=1)
    top_w, top_s = np.abs(np64(dw)).max(initial=0), 0.75 * np.abs(s0).max(initial=0)
    mag = 2 * top_s * share + 2 * abs(scale) * top_w * (mark[:, :E] + share)
    half = HALF_BF16 if z.dtype == torch.bfloat16 else U
    near(np64(d), d0, 400 * U * np.nan_to_num(mag) + half * np.abs(d0) + 1e-38, label + " d_logits")
    return ids, w, counts, loss, slope


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 7, 7), (33, 8, 2), (130, 16, 4), (65, 33, 5), (50, 64, 9),
                                   (40, 100, 8), (200, 128, 6), (77, 200, 3), (700, 256, 8), (31, 500, 10),
                                   (64, 512, 32), (21, 1001, 4), (300, 1024, 8)])
def test_route_sizes(fp8, T, E, k, dtype, renorm, scoring):
    z = logits_of(T, E, dtype, T * 1000 + E)
    check_route(fp8, z, k, scoring, renorm, 2.5 if scoring == "sigmoid" else 1.0, label=f"{T}x{E} k={k}")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(9001, 40), (9500, 200), (2049, 1000), (1500, 256)])
def test_route_many_rows(fp8, T, E, scoring):
    """One cluster of blocks in several turns, and more rows than one turn of
    the whole grid; an odd number of them, some masked."""
    g = np.random.default_rng(1)
    z = logits_of(T, E, torch.float32, 5)
    check_route(fp8, z, 4, scoring, True, mask=g.random(T) < 0.8, label="many rows")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [8, 100, 256])
def test_route_masks_and_extremes(fp8, E, dtype, renorm, scoring):
    """Closed experts, rows of -inf only, the type's lowest value, ties, zeros
    of both signs, rows whose scores all underflow, and NaN and infinities in
    masked rows."""
    z = logits_of(24, E, dtype, E)
    low = torch.finfo(dtype).min
    z[0] = -INF
    z[1] = -INF
    z[1, E // 2] = 1.0                     # one expert left for four slots
    z[2] = low
    z[3] = low
    z[3, 3] = -5.0
    z[4] = 0.25                            # all equal
    z[5] = 0.0
    z[5, 1::2] = -0.0                      # equal, whatever the sign
    z[6] = -200.0 - torch.arange(E) % 8    # sigmoid scores of 1e-87 and less
    z[7, :] = INF
    z[8, 2] = float("nan")
    z[9, 1::2] = -INF
    z[10] = -z[10].abs() - 90.0
    z[11] = torch.arange(E) % 4            # many ties
    mask = np.ones(24, bool)
    mask[[7, 8, 13]] = False
    check_route(fp8, z, 4, scoring, renorm, mask=mask, label=f"extremes E={E}")


def test_route_nan_shows(fp8):
    """A NaN logit beside others: never chosen, the row's shares and the loss
    are NaN, every other row is what it was."""
    z = logits_of(6, 32, torch.float32, 3)
    clean = fp8.route(z.cuda(), 4, balance=0.1)
    z[2, 7] = float("nan")
    ids, w, counts, loss, slope = check_route(fp8, z, 4, "softmax", True, label="nan")
    assert torch.isnan(loss).all() and torch.isnan(w[2]).all()
    other = [0, 1, 3, 4, 5]
    assert torch.equal(w[other], clean[1][other]) and torch.equal(ids[other], clean[0][other])


def test_route_empty_batch(fp8):
    z = torch.empty(0, 16, device="cuda")
    ids, w, counts, loss, slope = fp8.route(z, 2, balance=1.0)
    assert ids.shape == (0, 2) and counts.sum() == 0 and loss.item() == 0 and (slope == 0).all()
    assert fp8.route_backward(z, ids).shape == (0, 16)
    allmasked = fp8.route(torch.randn(5, 16, device="cuda"), 2, balance=1.0, mask=torch.zeros(5, dtype=torch.bool,
                                                                                           device="cuda"))
    assert (allmasked[0] == -1).all() and (allmasked[1] == 0).all() and allmasked[3].item() == 0


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [5, 64, 200])
def test_route_a_single_expert(fp8, E, dtype, scoring):
    """Renormalised, one chosen expert's weight is `scale` whatever the logits, so
    nothing comes back through it: the loss's gradient, however small beside
    d_weights, is all there is."""
    z = logits_of(300, E, dtype, 77)
    zd = z.cuda()
    ids, w, _, _, slope = fp8.route(zd, 1, scoring, True, 2.5, 1e-3)
    assert (w == 2.5).all()
    dw = torch.full((300, 1), 3.7, device="cuda")
    d = fp8.route_backward(zd, ids, dw, slope, None, scoring, True, 2.5)
    assert torch.equal(d, fp8.route_backward(zd, ids, None, slope, None, scoring, True, 2.5))
    zero = fp8.route_backward(zd, ids, dw, None, None, scoring, True, 2.5)
    assert (zero == 0).all()


def test_route_parts_of_the_gradient(fp8):
    """Only the weights', only the loss's, neither; and d_loss left out is 1."""
    z = logits_of(37, 48, torch.float32, 9)
    zd = z.cuda()
    ids, w, _, _, slope = fp8.route(zd, 6, "sigmoid", True, 2.0, 0.5)
    dw = torch.randn(37, 6, device="cuda")
    i0 = ids.cpu().numpy()
    for kw, rw, rs in ((dict(d_weights=dw), np64(dw), None), (dict(loss_grad=slope), None, np64(slope)), ({}, None, None)):
        got = fp8.route_backward(zd, ids, scoring="sigmoid", scale=2.0, **kw)
        want = ref.route_backward(np64(z), i0, rw, rs, 1.0, "sigmoid", True, 2.0)
        mag = 4 * (0 if rw is None else np.abs(rw).max()) + 2 * (0 if rs is None else np.abs(rs).max())
        near(np64(got), want, 400 * U * mag, str(list(kw)))


def test_route_same_bits_every_time(fp8):
    z = torch.randn(5000, 256, device="cuda")
    first = fp8.route(z, 8, balance=0.01)
    for _ in range(3):
        for a, b in zip(first, fp8.route(z, 8, balance=0.01)):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- group_rows

@pytest.mark.parametrize("n,G", [(0, 4), (1, 1), (31, 3), (64, 48), (4096, 256), (4097, 256), (12288, 1024), (20000, 7),
                                 (131072, 256), (300001, 1024), (600000, 3)])
@pytest.mark.parametrize("kind", ["random", "one", "none", "skewed"])
def test_group_rows(fp8, n, G, kind):
    g = np.random.default_rng(n + G)
    if kind == "random":
        ids = g.integers(-1, G + 1, n)
    elif kind == "one":
        ids = np.full(n, G - 1)
    elif kind == "none":
        ids = g.choice([-1, G, 2 ** 31 - 1, -2 ** 31], n)
    else:
        ids = np.minimum(g.geometric(0.3, n) - 1, G)
    ids = ids.astype(np.int32)
    offsets, order, slot = fp8.group_rows(torch.from_numpy(ids).cuda(), G)
    fp8.check()
    key = np.where((ids >= 0) & (ids < G), ids, G)
    o0 = np.argsort(key, kind="stable")
    f0 = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=G + 1)[:G])])
    s0 = np.empty(n, np.int64)
    s0[o0] = np.arange(n)
    assert np.array_equal(offsets.cpu().numpy(), f0)
    assert np.array_equal(order.cpu().numpy(), o0)
    assert np.array_equal(slot.cpu().numpy(), np.where(key < G, s0, -1))
    if n <= 20000:
        for a, b in zip((offsets, order, slot), ref.group_rows(ids, G)):
            assert np.array_equal(a.cpu().numpy(), b)


# -------------------------------------------------------------- combine_rows

def combine_case(T, k, H, n_extra, seed, drop=0.2):
    g = np.random.default_rng(seed)
    n = T * k + n_extra
    slot = g.permutation(T * k).reshape(T, k)
    slot = np.where(g.random((T, k)) < drop, -1, slot)
    # as group_rows leaves them: the rows in use come first
    used = np.sort(slot[slot >= 0])
    slot = np.where(slot >= 0, np.searchsorted(used, slot), -1).astype(np.int32)
    y = torch.randn(n, H, generator=torch.Generator().manual_seed(seed)).bfloat16()
    y[used.size:] = float("nan")           # rows that no slot names
    w = g.random((T, k)).astype(np.float32)
    w[slot < 0] = np.nan                   # weights of dropped entries
    return y, torch.from_numpy(w), torch.from_numpy(slot), used.size


@pytest.mark.parametrize("T,k,H,extra", [(1, 1, 8, 0), (1, 8, 7168, 0), (33, 2, 1024, 5), (7, 8, 1032, 0), (130, 9, 264, 3),
                                         (3, 32, 4096, 0), (513, 4, 2048, 700), (17, 10, 8200, 1)])
@pytest.mark.parametrize("with_base", [True, False])
def test_combine_rows(fp8, T, k, H, extra, with_base):
    y, w, slot, used = combine_case(T, k, H, extra, T + H)
    base = torch.randn(T, H, generator=torch.Generator().manual_seed(1)).bfloat16() if with_base else None
    bd = base.cuda() if with_base else None
    out = fp8.combine_rows(y.cuda(), w.cuda(), slot.cuda(), bd)
    want = ref.combine_rows(np64(y), np64(w), slot.numpy(), None if base is None else np64(base))
    mag = ref.combine_rows(np.abs(np64(y)), np64(w), slot.numpy(), None if base is None else np.abs(np64(base)))
    slack = (k + 2) * U * mag + HALF_BF16 * np.abs(want)
    near(np64(out), want, slack, "combine")
    if with_base:                          # in place on the base
        assert fp8.combine_rows(y.cuda(), w.cuda(), slot.cuda(), bd, out=bd) is bd
        assert torch.equal(bd, out)


@pytest.mark.parametrize("T,k,H,extra", [(1, 1, 8, 0), (1, 8, 7168, 0), (33, 2, 1024, 5), (7, 8, 1032, 0), (130, 9, 264, 3),
                                         (3, 32, 4096, 0), (513, 4, 2048, 700), (0, 2, 64, 9)])
def test_combine_gradient(fp8, T, k, H, extra):
    y, w, slot, used = combine_case(T, k, H, extra, T + H + 1)
    d_out = torch.randn(T, H, generator=torch.Generator().manual_seed(2)).bfloat16()
    offsets = torch.tensor([0, used], dtype=torch.int32, device="cuda")
    d_y = torch.full(y.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    got_y, got_w = fp8.combine_rows_backward(d_out.cuda(), y.cuda(), w.cuda(), slot.cuda(), offsets, d_y=d_y)
    fp8.check()
    want_y, want_w = ref.combine_rows_backward(np64(d_out), np64(y), np64(w), slot.numpy())
    _, mag = ref.combine_rows_backward(np.abs(np64(d_out)), np.abs(np64(y)), np64(w), slot.numpy())
    near(np64(got_y), want_y, (HALF_BF16 + U) * np.abs(want_y), "d_y")
    near(np64(got_w), want_w, (H / 128 + 24) * U * mag, "d_weights")
    assert (got_y[used:] == 0).all()


def test_combine_gradient_against_differences(fp8):
    """d_weights against central differences of the kernel's own forward: the
    output is linear in the weights, so a difference over a step of 1 is exact
    up to the two outputs' bf16 roundings."""
    T, k, H = 3, 2, 64
    y, w, slot, used = combine_case(T, k, H, 0, 11, drop=0.0)
    yd, wd, sd = y.cuda(), w.cuda(), slot.cuda()
    d_out = torch.randn(T, H).bfloat16().cuda()
    _, dw = fp8.combine_rows_backward(d_out, yd, wd, sd, torch.tensor([0, used], dtype=torch.int32, device="cuda"))
    for t in range(T):
        for j in range(k):
            up, dn = wd.clone(), wd.clone()
            up[t, j] += 0.5
            dn[t, j] -= 0.5
            a, b = fp8.combine_rows(yd, up, sd).double(), fp8.combine_rows(yd, dn, sd).double()
            diff = ((a - b) * d_out.double()).sum().item()
            slack = (HALF_BF16 * (a.abs() + b.abs()) * d_out.double().abs()).sum().item()
            assert abs(diff - dw[t, j].item()) <= 1.01 * slack


# ----------------------------------------------- refusals, streams, graphs

def test_refusals_on_device(fp8):
    d = "cuda"
    z = torch.randn(8, 16, device=d)
    ids = torch.zeros(8, 2, dtype=torch.int32, device=d)
    y = torch.randn(16, 64, device=d).bfloat16()
    w = torch.rand(8, 2, device=d)
    off = torch.zeros(3, dtype=torch.int32, device=d)
    big = torch.randn(5000, 256, device=d)
    bad = [
        (TypeError, lambda: fp8.route(z.half(), 2)),
        (ValueError, lambda: fp8.route(z.t(), 2)),
        (ValueError, lambda: fp8.route(z[:, ::2], 2)),
        (ValueError, lambda: fp8.route(z, 2, scoring="tanh")),
        (fp8.Fp8blError, lambda: fp8.route(z, 17)),
        (ValueError, lambda: fp8.route(z, 2, mask=torch.ones(9, dtype=torch.bool, device=d))),
        (TypeError, lambda: fp8.route(z, 2, mask=torch.ones(8, device=d))),
        (TypeError, lambda: fp8.route(z, 2, ids=ids.long())),
        (fp8.Fp8blError, lambda: fp8.route(big, 8, workspace=torch.empty(64, dtype=torch.uint8, device=d))),
        (fp8.Fp8blError, lambda: fp8.route(z, 2, weights=z.view(-1)[:16].view(8, 2))),
        (TypeError, lambda: fp8.route_backward(z, ids.float())),
        (ValueError, lambda: fp8.route_backward(z, ids, d_weights=w[:4])),
        (ValueError, lambda: fp8.route_backward(z, ids, loss_grad=torch.ones(15, device=d))),
        (ValueError, lambda: fp8.route_backward(z, ids, d_loss=torch.ones(1))),
        (TypeError, lambda: fp8.route_backward(z, ids, d_logits=z.bfloat16())),
        (TypeError, lambda: fp8.group_rows(ids.long(), 4)),
        (ValueError, lambda: fp8.group_rows(ids[:, :1], 4)),
        (ValueError, lambda: fp8.group_rows(ids, 4, offsets=off)),
        (fp8.Fp8blError, lambda: fp8.group_rows(ids, 1025)),
        (TypeError, lambda: fp8.combine_rows(y.float(), w, ids)),
        (ValueError, lambda: fp8.combine_rows(y, w[:4], ids)),
        (ValueError, lambda: fp8.combine_rows(y, w, ids, base=y)),
        (fp8.Fp8blError, lambda: fp8.combine_rows(y, w, ids, out=y[:8])),
        (fp8.Fp8blError, lambda: fp8.combine_rows(y[:, :60].contiguous(), w, ids)),
        (TypeError, lambda: fp8.combine_rows_backward(None, y, w, ids, off)),
        (ValueError, lambda: fp8.combine_rows_backward(y[:8], y, w, ids, off[:1])),
    ]
    for i, (exc, call) in enumerate(bad):
        with pytest.raises(exc):
            call()
    torch.cuda.synchronize()
    assert fp8.route(z, 2)[0].shape == (8, 2)
    fp8.check()


def test_other_stream_and_graphs_that_share_a_workspace(fp8):
    """The calls on a side stream, and two captured graphs that use one
    workspace, replayed in turn on changed inputs."""
    E, k, T, H = 64, 4, 3000, 256
    ws = torch.empty(max(fp8.route_workspace_bytes(T, E), fp8.group_rows_workspace_bytes(T * k, E)), dtype=torch.uint8,
                     device="cuda")
    zs = [torch.randn(T, E, device="cuda") for _ in range(2)]
    y = torch.randn(T * k, H, device="cuda").bfloat16()

    def step(z):
        ids, w, c, loss, slope = fp8.route(z, k, balance=0.01, workspace=ws)
        off, order, slot = fp8.group_rows(ids, E, workspace=ws)
        out = fp8.combine_rows(y, w, slot)
        d_y, d_w = fp8.combine_rows_backward(out, y, w, slot, off)
        return ids, w, c, loss, off, order, slot, out, d_y, d_w, fp8.route_backward(z, ids, d_w, slope)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for z in zs:
            step(z)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for z in zs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(z))
        graphs.append(g)
    for turn in range(2):
        for z in zs:
            z.copy_(torch.randn(T, E, device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for z, o in zip(zs, outs):
            for a, b in zip(step(z), o):
                assert torch.equal(a, b)
    fp8.check()


def test_the_expert_path(fp8):
    """Router, sort, quantization, both grouped linears and the weighted sum as
    an expert layer runs them, each step held to its definition on the inputs
    it really got; then the router's gradient through the weighted sum."""
    import oracle
    from tests.parity import check_gemm, u8
    T, E, k, K, N = 150, 8, 2, 256, 384
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    router = torch.randn(E, K, generator=g, device="cuda") * K ** -0.5
    wq, ws = fp8.quant_weight_ue8m0((torch.randn(E * N, K, generator=g, device="cuda") * 0.05).bfloat16())
    dq, ds = fp8.quant_weight_ue8m0((torch.randn(E * K, N, generator=g, device="cuda") * 0.05).bfloat16())
    wq, ws, dq, ds = wq.view(E, N, K), ws.view(E, N // 128, K // 128), dq.view(E, K, N), ds.view(E, K // 128, N // 128)
    logits = x.float() @ router.t()
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[-7:] = False                                     # a padded batch
    ids, w, counts, loss, slope = fp8.route(logits, k, balance=0.01, mask=mask)
    off, order, slot = fp8.group_rows(ids, E)
    assert torch.equal(off[1:] - off[:-1], counts)
    rows = x[(order // k).long()]                         # dropped entries behind off[-1]
    qa, sa = fp8.quant_act_ue8m0(rows)
    h = fp8.grouped_linear_ue8m0(qa, sa, wq, ws, off, y=torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda"))
    qh, sh = fp8.quant_act_ue8m0(torch.relu(h))
    y = torch.full((T * k, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    fp8.grouped_linear_ue8m0(qh, sh, dq, ds, off, y=y)
    out = fp8.combine_rows(y, w, slot, base=x)
    fp8.check()
    i0, w0, c0, _, _ = ref.route(np64(logits), k, mask=mask.cpu().numpy())
    f0, o0, s0 = ref.group_rows(i0, E)
    assert np.array_equal(ids.cpu().numpy(), i0) and np.array_equal(off.cpu().numpy(), f0)
    assert np.array_equal(order.cpu().numpy(), o0) and np.array_equal(slot.cpu().numpy(), s0)
    n = int(off[-1])
    R = oracle.grouped_linear_ue8m0(u8(qh), u8(sh), u8(dq), u8(ds), f0)
    check_gemm(y[:n].float().cpu().numpy(), R[:n], "down")
    want = ref.combine_rows(np.nan_to_num(np64(y)), np64(w), s0, np64(x))
    mag = ref.combine_rows(np.abs(np.nan_to_num(np64(y))), np64(w), s0, np.abs(np64(x)))
    near(np64(out), want, (k + 2) * U * mag + HALF_BF16 * np.abs(want), "out")
    assert torch.equal(out[-7:], x[-7:])                  # padded tokens keep the base
    d_y, d_w = fp8.combine_rows_backward(out, y, w, slot, off)
    d = fp8.route_backward(logits, ids, d_w, slope)
    fp8.check()
    assert torch.isfinite(d).all() and (d[-7:] == 0).all() and (d_y[n:] == 0).all()
    want = ref.route_backward(np64(logits), i0, np64(d_w), np64(slope))
    near(np64(d), want, 400 * U * (4 * np.abs(np64(d_w)).max() + 1), "router gradient")
