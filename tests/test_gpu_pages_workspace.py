"""One workspace of paged_tables_fork and paged_pages_compact for pools of several
sizes, and for both operations in any order: every call leaves it ready for the next."""
import numpy as np
import pytest
import torch

from tests.test_gpu_page_moves import Cache, check_compact, check_fork


def marks_are_zero(c):
    """The compaction's marks, two bytes a page behind the fork's word a page (which Cache.close looks at)."""
    at = 256 + 8 * 1024 + (4 * c.pages + 255) // 256 * 256
    assert int(c.workspace[at:at + 2 * c.pages].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("small,large", [(4000, 12000), (90, 91), (64, 30011), (11999, 12000), (40000, 70000)])
def test_pools_of_two_sizes(small, large):
    a, b = Cache([30] * 20, layers=1, pages=small, seed=1), Cache([30] * 20, layers=1, pages=large, seed=2)
    a.workspace = b.workspace
    for _ in range(2):
        for c in (a, b):
            check_compact(c)
            marks_are_zero(b)
            check_fork(c, list(range(0, 20, 3)))
        for c in (b, a):
            check_fork(c, [5, 5, 19])
            check_compact(c)
            marks_are_zero(b)
    a.close()
    b.close()


@pytest.mark.gpu
def test_pools_of_many_sizes_in_any_order():
    rng = np.random.default_rng(4)
    caches = [Cache([n] * 9, layers=2, hkv=1, pages=pages, seed=pages) for n, pages in
              ((5, 60), (70, 2048), (33, 2049), (16, 9001), (100, 33000), (400, 50000))]
    ws = torch.zeros(caches[-1].workspace.numel() + 1000, dtype=torch.uint8, device="cuda")  # no multiple of 256
    for c in caches:
        c.workspace = ws
    for i in rng.integers(0, 2 * len(caches), 60):
        c = caches[i // 2]
        check_compact(c) if i % 2 else check_fork(c, rng.integers(-1, 9, 7).tolist())
        marks_are_zero(caches[-1])
    for c in caches:
        c.close()


@pytest.mark.gpu
@pytest.mark.parametrize("layers,pages", [(1, 2000), (1, 9000), (40, 9000)])
def test_compactions_and_forks_after_one_another(layers, pages):
    """Other tables in each call: what a call left behind would show in the next."""
    c = Cache([100, 40, 7, 200], layers=layers, pages=pages, seed=layers)
    kept = c.tables, c.lens
    for step in range(3):
        c.tables, c.lens = kept
        check_compact(c)
        marks_are_zero(c)
        c.tables, c.lens = np.ascontiguousarray(kept[0][:, step:]), kept[1][step:]  # the others' pages are leaked
        check_compact(c)
        marks_are_zero(c)
        if step == 0:
            check_fork(c, [3, 1, 1, 0])
    c.close()
