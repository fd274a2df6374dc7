"""GPU parity of the low-rank adapters (lora_add) against their fp64
definition, alone and on top of the block linear.

Tolerance (u = 2^-24).  The inner product u_r adds K products of bf16 values
(exact in fp32) with at most K / 16 + 64 additions, each off by at most 2 u of
the magnitudes (the tensor core's adder may truncate): du_r = (K/16 + 64) 2u
sum|x a|.  u_r is multiplied as two bf16 terms, off by at most 2^-17 of it.
The outer sum adds 2 R products: 2 R 2u of the magnitudes.  The sum with y is
rounded once, half a bf16 step, 2^-8 of the result."""
import numpy as np
import pytest
import torch

from oracle import rows as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def make(M, N, K, R, L, seed, bare=0.1, spread=None):
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    ids = r.integers(0, L if spread is None else spread, M)
    ids = np.where(r.random(M) < bare, r.choice([-1, L + 3], M), ids).astype(np.int32)
    t = dict(x=torch.randn(M, K, generator=g).bfloat16(), a=(torch.randn(L, R, K, generator=g) * K ** -0.5).bfloat16(),
             b=(torch.randn(L, N, R, generator=g) * R ** -0.5).bfloat16(), y=torch.randn(M, N, generator=g).bfloat16(),
             scales=torch.rand(L, generator=g) + 0.5)
    return torch.from_numpy(ids), t


def bounds(t, ids, K, R):
    x, a, b, y = (np64(t[n]) for n in "xaby")
    s = np64(t["scales"]) if t["scales"] is not None else None
    want = ref.lora_add(y, x, a, b, ids.numpy(), s)
    mag = ref.lora_add(np.zeros_like(y), np.abs(x), np.abs(a), np.abs(b), ids.numpy(), s)
    return want, ((K / 16 + 64 + 2 * R) * 2 * U + 2.0 ** -17) * mag + (HALF_BF16 + U) * np.abs(want)


def run(fp8, t, ids, L, out=None):
    d = {k: None if v is None else v.cuda() for k, v in t.items()}
    off, order, _ = fp8.group_rows(ids.cuda(), L)
    out = d["y"] if out == "y" else out
    got = fp8.lora_add(d["y"], d["x"], d["a"], d["b"], off, order, scales=d["scales"], out=out)
    fp8.check()
    return got


def check(fp8, M, N, K, R, L, seed, **kw):
    ids, t = make(M, N, K, R, L, seed, **kw)
    got = run(fp8, t, ids, L)
    want, slack = bounds(t, ids, K, R)
    bad = ~(np.abs(np64(got) - want) <= slack)
    assert not bad.any(), (M, N, K, R, L, int(bad.sum()))
    none = (ids < 0) | (ids >= L)
    assert torch.equal(got.cpu()[none], t["y"][none])
    same = run(fp8, t, ids, L, out="y")
    assert torch.equal(same, got)
    return ids, t, got


@pytest.mark.parametrize("M,N,K,R,L", [(1, 28672, 4096, 16, 3), (16, 28672, 136, 16, 64), (9, 40, 14336, 8, 2),
                                       (1, 5000, 72, 128, 1), (1, 8, 8, 64, 5), (16, 2056, 2048, 16, 1)])
@pytest.mark.parametrize("bare", [0.0, 0.4, 1.0])
def test_a_few_rows(fp8, M, N, K, R, L, bare):
    """Both products in one launch: one cluster and several per tile, more
    columns than a cluster has warps for, fewer, K shorter than a cluster."""
    check(fp8, M, N, K, R, L, M + N + K, bare=bare)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("M", [1, 2, 17, 64, 65, 257, 300])
def test_ranks_and_rows(fp8, M, R):
    check(fp8, M, 264, 136, R, 3, M * 1000 + R)


@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("M,L", [(1025, 1), (1100, 3), (2051, 40)])
def test_ranks_of_long_batches(fp8, M, L, R):
    check(fp8, M, 200, 328, R, L, M * 1000 + R)


@pytest.mark.parametrize("R", [8, 32, 64, 72, 128])
@pytest.mark.parametrize("M,N,K,lengths", [
    (3000, 200, 328, [700, 1, 127, 128, 129, 1000, 255]),         # pieces of memory, some full tiles, some not
    (2500, 1096, 72, [512, 0, 512, 512, 300]),
    (4100, 72, 1544, [-3, 1024, -5, 1024, 900, 1000])])           # two requests of one adapter, apart
def test_requests_in_one_piece(fp8, M, N, K, lengths, R):
    """Requests of consecutive rows, as prompts come: their tiles go another way
    than scattered rows.  Negative lengths repeat the adapter of the request
    after next."""
    L = len(lengths)
    ids = np.full(M, -1, np.int32)
    at = 0
    for l, n in enumerate(lengths):
        ids[at:at + abs(n) * (100 if n < 0 else 1)] = (l + 2) % L if n < 0 else l
        at += abs(n) * (100 if n < 0 else 1)
    _, t = make(M, N, K, R, L, 50 + R)
    ids = torch.from_numpy(ids)
    got = run(fp8, t, ids, L)
    want, slack = bounds(t, ids, K, R)
    assert (np.abs(np64(got) - want) <= slack).all()
    assert torch.equal(run(fp8, t, ids, L, out="y"), got)


@pytest.mark.parametrize("M,N,K,R,L", [(1, 8, 8, 8, 1), (5, 8, 1000, 16, 2), (33, 1000, 8, 32, 4), (64, 4096, 1024, 16, 48),
                                       (512, 72, 2048, 64, 5), (700, 2056, 520, 16, 9), (1000, 136, 264, 128, 2),
                                       (2049, 512, 256, 8, 300), (48, 256, 128, 16, 1024), (1500, 64, 64, 16, 1024)])
def test_sizes(fp8, M, N, K, R, L):
    check(fp8, M, N, K, R, L, M + N + K)


@pytest.mark.parametrize("M,N,K,R,L", [(256, 136, 328, 128, 256), (256, 96, 2048, 64, 200), (41000, 72, 72, 8, 1),
                                       (39000, 8, 136, 72, 3)])
def test_more_tiles_than_blocks(fp8, M, N, K, R, L):
    """More tiles than the kernels' blocks work on at once."""
    ids, t = make(M, N, K, R, L, 40)
    got = run(fp8, t, ids, L)
    want, slack = bounds(t, ids, K, R)
    assert (np.abs(np64(got) - want) <= slack).all()


@pytest.mark.parametrize("M", [20, 400, 1100])
def test_few_adapters_in_use(fp8, M):
    """Most adapters without rows; every row without an adapter; every row on one."""
    check(fp8, M, 128, 128, 16, 100, 1, spread=2)
    check(fp8, M, 128, 128, 16, 4, 2, bare=1.0)
    check(fp8, M, 128, 128, 16, 1, 3, bare=0.0)


def test_no_scales_and_no_rows(fp8):
    ids, t = make(19, 128, 256, 16, 3, 8)
    t["scales"] = None
    want, slack = bounds(t, ids, 256, 16)
    assert (np.abs(np64(run(fp8, t, ids, 3)) - want) <= slack).all()
    empty = {k: v[:0].cuda() if k in "xy" else v.cuda() for k, v in t.items() if v is not None}
    got = fp8.lora_add(empty["y"], empty["x"], empty["a"], empty["b"], torch.zeros(4, dtype=torch.int32, device="cuda"),
                       torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert got.shape == (0, 128)


@pytest.mark.parametrize("M,R", [(40, 8), (40, 64), (300, 24), (300, 128), (1100, 8), (1100, 32)])
def test_adapters_and_rows_are_apart(fp8, M, R):
    """NaN and infinities in one adapter, in one row of x or of y stay there."""
    ids, t = make(M, 136, 264, R, 4, 12)
    clean = run(fp8, t, ids, 4)
    t["a"][1, :, 3] = float("nan")
    t["b"][2, 5] = float("inf")
    row = int(np.nonzero((ids == 0).numpy())[0][0])
    t["x"][row] = float("inf")
    t["y"][row + 1] = float("nan")
    got = run(fp8, t, ids, 4)
    apart = ((ids == 0) | (ids == 3) | (ids < 0) | (ids >= 4)).numpy()
    apart[[row, row + 1]] = False
    assert torch.equal(got[apart], clean[apart])
    assert torch.isnan(got[(ids == 1).numpy()]).all()
    cols = torch.arange(136) != 5
    two = (ids == 2).numpy()
    two[row + 1] = False
    assert torch.equal(got[two][:, cols], clean[two][:, cols])


def test_an_infinite_input_gives_what_the_sum_gives(fp8):
    """x = inf in one channel, A of one sign there: u = inf and the result +-inf
    by the sign of B (rank 8, padded inside to 16)."""
    ids, t = make(3, 64, 64, 8, 1, 13, bare=0.0)
    t["x"][1, 7] = float("inf")
    t["a"][0, :, 7] = 1.0
    t["b"][0] = t["b"][0].abs() + 0.125
    got = run(fp8, t, ids, 1)
    assert (got[1] == float("inf")).all() and torch.isfinite(got[[0, 2]]).all()


def test_same_bits_alone_and_in_a_batch_again(fp8):
    """The same call twice gives the same bits."""
    for M in (64, 1000, 1200):
        ids, t = make(M, 1024, 2048, 32, 6, 21)
        first = run(fp8, t, ids, 6)
        for _ in range(2):
            assert torch.equal(run(fp8, t, ids, 6), first)


def test_long_rows_past_32_bits(fp8):
    """y of more than 2^32 elements: the last rows are reached."""
    M, N, K, R = 32776, 131072, 16, 8
    x = torch.randn(M, K, device="cuda").bfloat16()
    y = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    a = torch.randn(1, R, K, device="cuda").bfloat16()
    b = torch.randn(1, N, R, device="cuda").bfloat16()
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-3:] = 0
    off, order, _ = fp8.group_rows(ids, 1)
    fp8.lora_add(y, x, a, b, off, order, out=y)
    fp8.check()
    want = (x[-3:].double() @ a[0].double().t()) @ b[0].double().t()
    # K = 16: products of bf16, u to 2^-17, the result to half a bf16 step
    mag = (x[-3:].double().abs() @ a[0].double().abs().t()) @ b[0].double().abs().t()
    assert ((y[-3:].double() - want).abs() <= HALF_BF16 * want.abs() + (2.0 ** -17 + 200 * U) * mag).all()
    assert (y[:-3].view(-1, N).abs().amax(1) == 0).all()


def test_order_with_rows_outside(fp8):
    """Rows named outside [0, M) are skipped, offsets are clamped."""
    ids, t = make(20, 64, 64, 16, 2, 30, bare=0.0)
    off, order, _ = fp8.group_rows(ids.cuda(), 2)
    d = {k: v.cuda() for k, v in t.items()}
    good = fp8.lora_add(d["y"], d["x"], d["a"], d["b"], off, order, scales=d["scales"])
    bad = order.clone()
    bad[3], bad[11] = -5, 20
    off2 = off.clone()
    off2[0], off2[2] = -9, 1000
    out = torch.full_like(d["y"], 7.0)
    fp8.lora_add(d["y"], d["x"], d["a"], d["b"], off2, bad, scales=d["scales"], out=out)
    fp8.check()
    gone = order[[3, 11]].long()
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[gone] = False
    assert torch.equal(out[keep], good[keep]) and (out[gone] == 7.0).all()


def test_refusals_on_device(fp8):
    ids, t = make(20, 64, 64, 16, 2, 31)
    d = {k: v.cuda() for k, v in t.items()}
    off, order, _ = fp8.group_rows(ids.cuda(), 2)
    y, x, a, b, s = d["y"], d["x"], d["a"], d["b"], d["scales"]
    for exc, call in (
            (TypeError, lambda: fp8.lora_add(y, x.float(), a, b, off, order)),
            (ValueError, lambda: fp8.lora_add(y[:, :32], x, a, b, off, order)),
            (ValueError, lambda: fp8.lora_add(y, x, a[0], b, off, order)),
            (ValueError, lambda: fp8.lora_add(y, x, a, b[:1], off, order)),
            (ValueError, lambda: fp8.lora_add(y, x, a, b.transpose(1, 2), off, order)),
            (ValueError, lambda: fp8.lora_add(y, x, a, b, off[:2], order)),
            (ValueError, lambda: fp8.lora_add(y, x, a, b, off, order[:5])),
            (TypeError, lambda: fp8.lora_add(y, x, a, b, off.long(), order)),
            (TypeError, lambda: fp8.lora_add(y, x, a, b, off, order, scales=s.bfloat16())),
            (fp8.Fp8blError, lambda: fp8.lora_add(y, x, a, b, off, order, out=x)),
            (fp8.Fp8blError, lambda: fp8.lora_add(y, x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), off, order)),
            (TypeError, lambda: fp8.lora_add(y, x, None, b, off, order))):
        with pytest.raises(exc):
            call()
    fp8.lora_add(y, x, a, b, off, order)
    fp8.check()


@pytest.mark.parametrize("M", [5, 64, 300, 1100])
def test_beside_the_block_linear(fp8, M):
    """The shared projection and the adapters on top of it, on a side stream and
    as a captured graph that is replayed on new inputs."""
    N, K, R, L = 256, 384, 16, 4
    ids, t = make(M, N, K, R, L, M)
    d = {k: v.cuda() for k, v in t.items()}
    q_w, s_w = fp8.quant_weight((torch.randn(N, K, device="cuda") * 0.05).bfloat16())
    off, order, _ = fp8.group_rows(ids.cuda(), L)
    ws = torch.empty(max(1, fp8.lora_add_workspace_bytes(M, N, K, R, L)), dtype=torch.uint8, device="cuda")

    def step():
        y = fp8.block_linear_fused(d["x"], q_w, s_w)
        return y.clone(), fp8.lora_add(y, d["x"], d["a"], d["b"], off, order, scales=d["scales"], out=y, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        base, out = step()
    for turn in range(2):
        d["x"].copy_(torch.randn(M, K, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        t["x"], t["y"] = d["x"].cpu(), base.cpu()
        want, slack = bounds(t, ids, K, R)
        assert (np.abs(np64(out) - want) <= slack).all()
        again, mine = step()
        assert torch.equal(again, base) and torch.equal(mine, out)
    fp8.check()
