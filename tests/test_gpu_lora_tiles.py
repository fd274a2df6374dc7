"""The long form of the adapters (lora_add) where a block or a cluster goes on
from one 128-row tile to the next: full tiles of consecutive rows, which come
and go by TMA, full tiles of scattered rows and partial ones, which do not, in
every order.  Every case first works out, from the tiles and the launch sizes,
which steps it takes, and asserts that they are the ones it is there for.

Tolerance: as derived for the other tests of lora_add."""
import numpy as np
import pytest
import torch

from tests.test_gpu_lora import bounds, make, np64, run

pytestmark = pytest.mark.gpu
ROWS, COLS = 128, 64    # of a tile, of the expand's chunks


@pytest.fixture(scope="module")
def fp8():
    import fine_grained_block_token_b200 as m
    return m


def requests(lengths, adapters, scattered=()):
    """Rows of consecutive requests, adapter i % adapters each; two requests in
    `scattered` share their rows in turn."""
    ids = np.concatenate([np.full(n, i % adapters) for i, n in enumerate(lengths)]).astype(np.int32)
    start = np.concatenate([[0], np.cumsum(lengths)])
    for i, j in scattered:
        at = np.r_[start[i]:start[i + 1], start[j]:start[j + 1]]
        ids[at[::2]], ids[at[1::2]] = i % adapters, j % adapters
    return ids


def tiles_of(ids, L):
    """'T' for a full tile of consecutive rows, 'F' for a full one of scattered
    rows, 'P' for a partial one, in the order of the kernels' tile numbers."""
    out = []
    for l in range(L):
        rows = np.nonzero(ids == l)[0]
        for t in range(0, rows.size, ROWS):
            r = rows[t:t + ROWS]
            out.append("P" if r.size < ROWS else "T" if r[-1] - r[0] == ROWS - 1 else "F")
    return out


def expand_steps(kinds, N, R):
    """The steps from one tile to the next that the expand's blocks take
    (every adapter's tiles, in place: no rows to copy)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    blocks, chunks = sms * (1 if R > 64 else 2), -(-N // COLS)
    total = len(kinds) * chunks
    blocks = min(blocks, total)
    team = min(blocks // len(kinds), chunks)
    if 10 * team * len(kinds) >= 9 * blocks:
        return set()
    steps = set()
    for b in range(blocks):
        lo, hi = total * b // blocks, total * (b + 1) // blocks
        mine = [kinds[t] for t in range(lo // chunks, -(-hi // chunks))] if hi > lo else []
        steps |= {a + b for a, b in zip(mine, mine[1:])}
    return steps


def compare(fp8, ids, t, K, R, L):
    ids = torch.from_numpy(ids)
    got = run(fp8, t, ids, L)
    want, slack = bounds(t, ids, K, R)
    bad = ~(np.abs(np64(got) - want) <= slack)
    assert not bad.any(), (int(bad.sum()), np.unique(np.nonzero(bad)[0] // ROWS)[:10])
    for _ in range(2):
        assert torch.equal(run(fp8, t, ids, L, out="y"), got)


@pytest.mark.parametrize("R", [8, 32, 64, 72, 128])
@pytest.mark.parametrize("N", [136, 584])
def test_expand_goes_from_tile_to_tile(fp8, N, R):
    """Blocks of the expand with several runs: the copies' warp hands its slots
    over between every pair of kinds.  One tile for every cluster of the shrink."""
    K, L = 72, 12
    g = np.random.default_rng(R)
    lengths = [int(n) for n in g.integers(1, 12, 60) * ROWS + np.where(g.random(60) < 0.5, 0, g.integers(1, 127, 60))]
    while len(tiles_of(requests(lengths, L), L)) > 225:
        lengths.pop()
    ids = requests(lengths, L, [(0, 1), (14, 15)])
    kinds = tiles_of(ids, L)
    assert expand_steps(kinds, N, R) >= {"TT", "TP", "PT", "TF", "FT", "FF"}
    _, t = make(ids.size, N, K, R, L, 70 + R)
    compare(fp8, ids, t, K, R, L)


def shrink_steps(kinds, clusters):
    """The steps from one tile to the next that the shrink's clusters take."""
    steps = set()
    for c in range(clusters):
        mine = kinds[c::clusters]
        steps |= {a + b for a, b in zip(mine, mine[1:])}
    return steps


@pytest.mark.parametrize("R", [8, 32, 64, 128])
@pytest.mark.parametrize("K", [72, 520])
def test_shrink_goes_from_tile_to_tile(fp8, K, R):
    """Blocks of the shrink that take several tiles: the ring that held the sums
    of one is filled again by TMA or by plain copies."""
    N, L = 72, 7
    g = np.random.default_rng(R + K)
    lengths = [int(n) for n in g.integers(1, 30, 46) * ROWS + np.where(g.random(46) < 0.5, 0, g.integers(1, 127, 46))]
    ids = requests(lengths, L, [(0, 1), (9, 10), (25, 26), (30, 31)])
    kinds = tiles_of(ids, L)
    # too many for clusters of more than one block: two blocks per SM
    clusters = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    assert shrink_steps(kinds, clusters) >= {"TT", "TF", "FT", "FF", "TP", "PT"}
    _, t = make(ids.size, N, K, R, L, 80 + R)
    compare(fp8, ids, t, K, R, L)


@pytest.mark.parametrize("R", [8, 64, 128])
@pytest.mark.parametrize("M,K,parts", [(7680, 520, 2), (4000, 1160, 4), (2100, 1560, 6)])
def test_shrink_clusters_go_from_tile_to_tile(fp8, M, K, parts, R):
    """The same where the blocks of a cluster share K, at least 256 each: the ring
    also held what the other blocks read.  Adapters with a few rows lie between
    two of long requests, so that whatever number of clusters the chip holds
    some go from the first to the second."""
    N, L = 72, 400
    at_once = 2 * torch.cuda.get_device_properties(0).multi_processor_count // parts
    first, last = M * 3 // 8 // ROWS * ROWS, M // 4 // ROWS * ROWS
    few = at_once * 7 // 8 - 1
    ids = np.zeros(M, np.int32)
    ids[first:M - last] = 1 + np.arange(M - first - last) % few
    ids[M - last:] = L - 1
    kinds = tiles_of(ids, L)
    assert K // 256 == parts and len(kinds) > at_once
    for clusters in range(at_once * 7 // 8, at_once + 1):
        assert "TT" in shrink_steps(kinds, clusters)
    _, t = make(M, N, K, R, L, 90 + R)
    compare(fp8, ids, t, K, R, L)


@pytest.mark.parametrize("R", [16, 72])
@pytest.mark.parametrize("parts", range(1, 9))
def test_clusters_of_every_size(fp8, parts, R):
    """One part of K, at least 256 deep, for every block of a cluster: 1 to 8 blocks,
    all of whose shares of the rows are added up, the last one's shorter too."""
    M, N, K, L = 2100, 136, 256 * parts + 200, 3
    ids, t = make(M, N, K, R, L, 100 + parts)
    ids[:700] = 1
    compare(fp8, ids.numpy(), t, K, R, L)
