"""The row and adapter calls beside one another: two streams at once, graphs
that share a workspace, and tensors of more than 2^31 and 2^32 elements."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


def adapters(M, N, K, R, L, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ids = (torch.arange(M, device="cuda") * (L + 1) // M).int()          # the last request has no adapter
    return dict(y=rnd(M, N), x=rnd(M, K), a=rnd(L, R, K), b=rnd(L, N, R)), ids


# one launch, 16-row tiles, long batches with clusters of several sizes, with several tiles a block
CASES = [(9, 4096, 1024, 16, 4), (200, 2056, 1032, 32, 9), (3000, 1096, 2056, 16, 3), (2500, 520, 520, 128, 5),
         (45000, 136, 72, 64, 3)]


def test_two_streams_at_once(fp8):
    """Each stream runs every call in another order, with workspaces of its own;
    the bits are those of the calls one by one."""
    work = []
    for i, (M, N, K, R, L) in enumerate(CASES):
        t, ids = adapters(M, N, K, R, L, i)
        off, order, _ = fp8.group_rows(ids, L)
        work.append(lambda t=t, off=off, order=order: (fp8.lora_add(**t, offsets=off, order=order),))
    for i, (T, E) in enumerate(((1, 256), (500, 64), (9000, 40))):
        z = torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(50 + i), device="cuda")
        work.append(lambda z=z: fp8.route(z, 4, "sigmoid", balance=0.01))
        work.append(lambda z=z, E=E: fp8.group_rows(fp8.route(z, 4)[0], E))
    alone = [f() for f in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(5):
        got = {}
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in range(len(work)):
            for j, s in enumerate(streams):
                at = (i * (1 + 2 * j) + 3 * j + turn) % len(work)
                with torch.cuda.stream(s):
                    got[j, at] = work[at]()
        torch.cuda.synchronize()
        fp8.check()
        for (_, at), outs in got.items():
            for a, b in zip(outs, alone[at]):
                assert torch.equal(a, b), at
        assert len(got) == 2 * len(work)


@pytest.mark.parametrize("M,N,K,R,L", CASES)
def test_graphs_that_share_the_adapters_workspace(fp8, M, N, K, R, L):
    ws = torch.empty(max(16, fp8.lora_add_workspace_bytes(M, N, K, R, L)), dtype=torch.uint8, device="cuda")
    states, graphs, outs = [], [], []
    side = torch.cuda.Stream()
    for seed in (1, 2):
        t, ids = adapters(M, N, K, R, L, seed)
        off, order, _ = fp8.group_rows(ids, L)
        out = torch.empty_like(t["y"])
        call = lambda t=t, off=off, order=order, out=out: fp8.lora_add(  # noqa: E731
            **t, offsets=off, order=order, out=out, workspace=ws)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        states.append((t, off, order))
        graphs.append(g)
        outs.append(out)
    for turn in range(3):
        for t, _, _ in states:
            t["x"].copy_(torch.randn_like(t["x"]))
        ws.fill_(0xFF)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (t, off, order), out in zip(states, outs):
            assert torch.equal(fp8.lora_add(**t, offsets=off, order=order), out)
    fp8.check()


def test_weighted_sum_past_32_bits(fp8):
    """y of more than 2^32 elements: the last rows are read and written."""
    n, H, T, k = 600_000, 7168, 5, 3
    y = torch.zeros(n, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.randn(T * k, H, device="cuda").bfloat16()
    y[n - T * k:] = rows
    slot = torch.arange(n - T * k, n, dtype=torch.int32, device="cuda").view(T, k)
    w = torch.rand(T, k, device="cuda")
    near = torch.arange(T * k, dtype=torch.int32, device="cuda").view(T, k)
    out = fp8.combine_rows(y, w, slot)
    assert torch.equal(out, fp8.combine_rows(rows, w, near))
    d_y, d_w = fp8.combine_rows_backward(out, y, w, slot, torch.tensor([0, n], dtype=torch.int32, device="cuda"), d_y=None)
    e_y, e_w = fp8.combine_rows_backward(out, rows, w, near, torch.tensor([0, T * k], dtype=torch.int32, device="cuda"))
    assert torch.equal(d_y[n - T * k:], e_y) and torch.equal(d_w, e_w)
    # only the rows behind the last named one are written as zeros
    d_y.fill_(1.0)
    fp8.combine_rows_backward(out, y, w, near, torch.tensor([0, n - 7], dtype=torch.int32, device="cuda"), d_y=d_y)
    assert (d_y[n - 7:] == 0).all() and (d_y[n - 50:n - 7] == 1).all()


def test_router_past_32_bits(fp8):
    """Logits of more than 2^31 elements: the last rows are what they are alone."""
    T, E, k = (1 << 21) + 5, 1024, 4
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(64, E, device="cuda").bfloat16()
    z[-64:] = last
    ids, w, counts, _, _ = fp8.route(z, k, "sigmoid")
    few = fp8.route(last, k, "sigmoid")
    assert torch.equal(ids[-64:], few[0]) and torch.equal(w[-64:], few[1])
    assert int(counts.sum()) == T * k and (ids[:-64] == torch.arange(k, device="cuda")).all()
    dw = torch.randn(T, k, device="cuda")
    d = fp8.route_backward(z, ids, dw, None, None, "sigmoid")
    assert torch.equal(d[-64:], fp8.route_backward(last, few[0], dw[-64:].contiguous(), None, None, "sigmoid"))
    fp8.check()
