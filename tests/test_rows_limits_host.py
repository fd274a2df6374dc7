"""Host-side checks of the row calls' limits (no GPU needed)."""
import ctypes

import pytest

from tests.test_rows_host import AT, I64, SHAPE, SZ, V, _call


@pytest.fixture(scope="module")
def lib():
    from fine_grained_block_token_b200 import build
    return ctypes.CDLL(build.build())


def test_adapter_tiles_are_counted_in_32_bits(lib):
    """Offsets that go up and down may name every row (L + 1) / 2 times over; the
    tiles they make still have to be countable."""
    def status(M, L):
        return _call(lib.fp8bl_lora_add, [V] * 8 + [I64] * 5 + [V, SZ, V],
                     [*AT[:8], M, 8, 8, 8, L, None, 0, None])
    for M, L in ((1 << 30, 1024), (1 << 28, 1024), (1 << 30, 128)):
        assert (L + 1) * M > 1 << 37 and status(M, L) == SHAPE
    lib.fp8bl_lora_add_workspace_bytes.argtypes, lib.fp8bl_lora_add_workspace_bytes.restype = [I64] * 5, SZ
    assert lib.fp8bl_lora_add_workspace_bytes(1 << 30, 8, 8, 8, 128) == 0
    assert lib.fp8bl_lora_add_workspace_bytes(1 << 30, 8, 8, 8, 127) > 0
    assert lib.fp8bl_lora_add_workspace_bytes(1 << 26, 8, 8, 8, 1024) > 0


def test_the_size_error_names_the_linears_multiple(lib):
    """The most frequent wrong size of the linears stays in the message."""
    lib.fp8bl_status_string.restype = ctypes.c_char_p
    assert b"multiples of 128" in lib.fp8bl_status_string(SHAPE)


@pytest.mark.parametrize("E,rows", [(8, 128), (16, 128), (64, 128), (100, 64), (256, 32), (512, 16), (1024, 8)])
def test_the_router_takes_the_whole_gpu_beyond_one_turn_of_a_cluster(lib, E, rows):
    """A block has `rows` rows in flight; what one cluster of eight cannot take at
    once goes to all SMs, with a workspace for their sums."""
    lib.fp8bl_route_workspace_bytes.argtypes, lib.fp8bl_route_workspace_bytes.restype = [I64] * 2, SZ
    for T in (1, rows, rows + 1, 8 * rows):
        assert lib.fp8bl_route_workspace_bytes(T, E) == 0
    assert lib.fp8bl_route_workspace_bytes(8 * rows + 1, E) == 9 * (8 * E + 4)
    assert lib.fp8bl_route_workspace_bytes(32 * rows, E) == 32 * (8 * E + 4)
