"""Host-side checks of the router, row and adapter calls (no GPU needed):
every refusal comes back as its status before the device is touched, and the
workspace sizes follow their documented bounds."""
import ctypes

import pytest
import torch

I64, INT, F32, V, SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
NULL, SHAPE, ALIGN, OVERLAP = 1, 2, 3, 8
AT = [V(0x10000000 * (i + 1)) for i in range(16)]   # far apart, aligned


@pytest.fixture(scope="module")
def lib():
    from fine_grained_block_token_b200 import build
    return ctypes.CDLL(build.build())


def _call(f, types, args):
    f.argtypes, f.restype = types, INT
    return f(*args)


def _route(lib, **k):
    a = dict(logits=AT[0], type=1, T=4, E=16, k=2, scoring=0, renorm=1, scale=1.0, balance=0.0, mask=None,
             ids=AT[1], weights=AT[2], counts=AT[3], loss=AT[4], loss_grad=AT[5], ws=None, wsb=0, st=None)
    assert not set(k) - set(a)
    a.update(k)
    return _call(lib.fp8bl_route, [V, INT, I64, I64, I64, INT, INT, F32, F32, V, V, V, V, V, V, V, SZ, V],
                 list(a.values()))


def test_route_refusals(lib):
    for bad in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=64, k=33),
                dict(type=2), dict(scoring=2), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(balance=float("nan"))):
        assert _route(lib, **bad) == SHAPE, bad
    for name in ("logits", "ids", "weights", "counts"):
        assert _route(lib, **{name: None}) == NULL, name
    assert _route(lib, T=0, logits=None, ids=None, weights=None, counts=None) == NULL  # counts are written
    assert _route(lib, logits=V(0x10000008)) == ALIGN
    for name in ("ids", "weights", "counts", "loss", "loss_grad"):
        assert _route(lib, **{name: V(0x90000002)}) == ALIGN, name
        assert _route(lib, **{name: V(0x10000004)}) == OVERLAP, name    # into the logits
    assert _route(lib, weights=V(AT[1].value + 4)) == OVERLAP
    assert _route(lib, mask=V(0x20000001)) == OVERLAP                    # the mask inside ids


def test_route_backward_refusals(lib):
    def call(**k):
        a = dict(logits=AT[0], type=0, ids=AT[1], dw=AT[2], lg=AT[3], dl=AT[4], T=4, E=16, k=2, scoring=1, renorm=1,
                 scale=1.0, d=AT[5], st=None)
        a.update(k)
        return _call(lib.fp8bl_route_backward, [V, INT, V, V, V, V, I64, I64, I64, INT, INT, F32, V, V],
                     list(a.values()))
    for bad in (dict(T=-1), dict(E=1025), dict(k=0), dict(k=17), dict(type=-1), dict(scoring=-1),
                dict(scale=float("inf"))):
        assert call(**bad) == SHAPE, bad
    assert call(T=0, logits=None, ids=None, d=None) == 0
    for name in ("logits", "ids", "d"):
        assert call(**{name: None}) == NULL, name
    assert call(d=V(0x90000008)) == ALIGN
    for i in range(5):
        assert call(d=AT[i]) == OVERLAP, i


def test_group_refusals(lib):
    def call(**k):
        a = dict(ids=AT[0], n=100, G=8, offsets=AT[1], order=AT[2], slot=AT[3], ws=None, wsb=0, st=None)
        a.update(k)
        return _call(lib.fp8bl_group_rows, [V, I64, I64, V, V, V, V, SZ, V], list(a.values()))
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(G=0), dict(G=1025)):
        assert call(**bad) == SHAPE, bad
    for name in ("ids", "offsets", "order", "slot"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: V(0x90000001)}) == ALIGN, name
    for name in ("offsets", "order", "slot"):
        assert call(**{name: V(AT[0].value + 396)}) == OVERLAP, name
    assert call(slot=AT[2]) == OVERLAP


def test_combine_refusals(lib):
    def fwd(**k):
        a = dict(y=AT[0], w=AT[1], slot=AT[2], base=None, out=AT[3], T=4, n=8, k=2, H=64, st=None)
        a.update(k)
        return _call(lib.fp8bl_combine_rows, [V] * 5 + [I64] * 4 + [V], list(a.values()))

    def back(**k):
        a = dict(d_out=AT[0], y=AT[1], w=AT[2], slot=AT[3], used=AT[4], d_y=AT[5], d_w=AT[6], T=4, n=8, k=2, H=64,
                 st=None)
        a.update(k)
        return _call(lib.fp8bl_combine_rows_backward, [V] * 7 + [I64] * 4 + [V], list(a.values()))
    for call in (fwd, back):
        for bad in (dict(T=-1), dict(n=-1), dict(k=0), dict(k=33), dict(H=0), dict(H=12), dict(T=1 << 30, H=8192)):
            assert call(**bad) == SHAPE, bad
        for name in ("y", "w", "slot"):
            assert call(**{name: None}) == NULL, name
        assert call(y=V(0x90000008)) == ALIGN
    assert fwd(T=0, y=None, w=None, slot=None, out=None) == 0
    assert back(T=0, n=0, d_out=None, y=None, w=None, slot=None, used=None, d_y=None, d_w=None) == 0
    assert fwd(out=None) == NULL and back(used=None) == NULL and back(d_w=None) == NULL
    for i in range(3):
        assert fwd(out=AT[i]) == OVERLAP
    assert fwd(base=V(AT[3].value + 16)) == OVERLAP    # part of out, not out itself
    for i in range(5):
        assert back(d_y=AT[i]) == OVERLAP and back(d_w=AT[i]) == OVERLAP
    assert back(d_w=AT[5]) == OVERLAP


def test_lora_refusals(lib):
    def call(**k):
        a = dict(x=AT[0], a=AT[1], b=AT[2], scales=AT[3], offsets=AT[4], order=AT[5], y=AT[6], out=AT[7], M=4, N=64,
                 K=64, R=16, L=2, ws=None, wsb=0, st=None)
        a.update(k)
        return _call(lib.fp8bl_lora_add, [V] * 8 + [I64] * 5 + [V, SZ, V], list(a.values()))
    for bad in (dict(M=-1), dict(N=0), dict(N=60), dict(K=0), dict(K=100), dict(R=0), dict(R=12), dict(R=136),
                dict(L=0), dict(L=1025)):
        assert call(**bad) == SHAPE, bad
    assert call(M=0, x=None, y=None, out=None) == 0
    for name in ("x", "a", "b", "offsets", "order", "y", "out"):
        assert call(**{name: None}) == NULL, name
        assert call(**{name: V(0x91000002)}) == ALIGN, name
    for i in range(6):
        assert call(out=AT[i]) == OVERLAP, i
    assert call(out=V(AT[6].value + 16)) == OVERLAP    # part of y, not y itself


def test_workspace_sizes(lib):
    """Never fail: 0 for sizes the call refuses, and bounded as documented."""
    def size(name, *a):
        f = getattr(lib, name)
        f.argtypes, f.restype = [I64] * len(a), SZ
        return f(*a)
    assert size("fp8bl_route_workspace_bytes", 1, 256) == 0
    for T, E in ((-1, 8), (8, 0), (8, 2000)):
        assert size("fp8bl_route_workspace_bytes", T, E) == 0
    assert 0 < size("fp8bl_route_workspace_bytes", 1 << 20, 1024) <= 256 * (1024 * 8 + 4)
    assert size("fp8bl_group_rows_workspace_bytes", 64, 48) == 0
    assert 0 < size("fp8bl_group_rows_workspace_bytes", 1 << 30, 1024) <= 256 * 1025 * 4
    assert size("fp8bl_group_rows_workspace_bytes", 100000, 1025) == 0
    assert size("fp8bl_route_workspace_bytes", 0, 8) == 0
    assert size("fp8bl_group_rows_workspace_bytes", 0, 8) == 0
    assert size("fp8bl_lora_add_workspace_bytes", 0, 128, 64, 16, 2) == 0
    assert size("fp8bl_lora_add_workspace_bytes", 16, 4096, 4096, 16, 4) == 0   # one launch
    assert size("fp8bl_lora_add_workspace_bytes", 64, 4096, 4096, 16, 4) > 0
    assert size("fp8bl_lora_add_workspace_bytes", 64, 100, 64, 16, 2) == 0
    assert size("fp8bl_lora_add_workspace_bytes", 5000, 4096, 14336, 128, 64) <= 64 << 20


def test_host_tensors_refused():
    import fine_grained_block_token_b200 as fp8
    z, i = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    y, w = torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(4, 2)
    o = torch.zeros(3, dtype=torch.int32)
    ab = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16)
    for call in (lambda: fp8.route(z, 2), lambda: fp8.route_backward(z, i), lambda: fp8.group_rows(i, 2),
                 lambda: fp8.combine_rows(y, w, i), lambda: fp8.combine_rows_backward(y[:4], y, w, i, o),
                 lambda: fp8.lora_add(y, y, *ab, o, torch.zeros(8, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
