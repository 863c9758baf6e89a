"""Forks and compactions that are one cluster, in pools of up to 12 chunks (of 2048
pages), and by grids on the other side of that border. Which call is which
is test_page_launches.py's."""
import numpy as np
import pytest

from tests.test_gpu_page_moves import Cache, check_compact, check_fork
from tests.test_gpu_pages_workspace import marks_are_zero

CHUNK, MOST = 2048, 12
POOLS = [CHUNK + 1, 3 * CHUNK, 6 * CHUNK + 5, 9 * CHUNK - 1, 11 * CHUNK, MOST * CHUNK - 1, MOST * CHUNK, MOST * CHUNK + 1]


@pytest.mark.gpu
@pytest.mark.parametrize("pages", POOLS)
@pytest.mark.parametrize("lens,parents", [
    ([1] * 200, list(range(0, 200, 3))),                 # a third goes on, the others' pages come back from every chunk
    ([70] * 150, [7, 7, 149, 3, 3, 3, -1] * 15),         # copies, and most of the sequences dropped
    ([16 * 300, 33, 16 * 40 + 1], [2, 0, 2, 2])])
def test_forks(pages, lens, parents):
    c = Cache(lens, layers=1, hkv=1, pages=pages, seed=pages)
    assert len(parents) + (len(lens) + len(parents)) * -(-c.tables.shape[2] // 128) <= 640
    for _ in range(2):
        check_fork(c, parents)
        check_fork(c, [])  # everything is given back
    c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("pages", POOLS)
@pytest.mark.parametrize("held", [1, 3, 8, 14])  # sixteenths of the pool
def test_compactions(pages, held):
    rng = np.random.default_rng(pages + held)
    blocks = pages // CHUNK * 128  # whole parts of the rows: fewest pieces of work
    c = Cache([1], layers=1, hkv=1, pages=pages, seed=held)
    perm = rng.permutation(pages).astype(np.int32)
    c.tables = perm[:held * blocks].reshape(1, held, blocks)
    c.lens = np.full(held, 16 * blocks, np.int32)
    c.lens[0] -= 3
    c.shares = np.zeros(pages, np.int32)
    c.shares[perm[:50]] = rng.integers(1, 9, 50)
    c.free, c.head = perm[held * blocks:], 0
    if pages <= MOST * CHUNK:
        assert held * -(-blocks // 128) + -(-len(c.free) // 128) <= 256
    for _ in range(2):
        check_compact(c)
        marks_are_zero(c)
    c.free = rng.permutation(c.free)[:len(c.free) // 3]  # the others are somebody else's
    check_compact(c)
    c.close()
