"""paged_tables_build refuses arrays that overlap one that it writes: every CTA
reads all lengths while the first one writes the new ones."""
import ctypes

import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

BATCH, LAYERS, FREE, BLOCKS, CAPACITY = 4, 2, 9, 5, 7
# argument index and size in int32 of what is read and what is written
READ = {"start_pos": (1, BATCH), "new_tokens": (2, BATCH), "free_pages": (5, FREE), "free_head": (7, 1)}
WRITTEN = {"free_head_out": (8, 1), "block_tables": (9, LAYERS * BATCH * BLOCKS), "cu_tokens": (11, BATCH + 1),
           "seq_lens": (12, BATCH), "positions": (13, CAPACITY), "slot_map": (14, LAYERS * CAPACITY)}
SHAPE = {"block_tables": (LAYERS, BATCH, BLOCKS), "slot_map": (LAYERS, CAPACITY)}
PAIRS = [(w, o) for w in WRITTEN for o in {**READ, **WRITTEN} if w != o]


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses that are no memory; no launch can happen here")
def test_the_library_refuses_overlapping_arrays():
    pool = ctypes.create_string_buffer(4096)
    at = {name: 1 << 20 | i << 12 for i, name in enumerate({**READ, **WRITTEN})}

    def call(**moved):
        args = [ctypes.addressof(pool), 0, 0, BATCH, LAYERS, 0, FREE, 0, 0, 0, BLOCKS, 0, 0, 0, 0, CAPACITY, None]
        for name, (i, _) in {**READ, **WRITTEN}.items():
            args[i] = {**at, **moved}[name]
        return pkv.lib().paged_tables_build(*args)

    assert call() == -5  # not refused: the launch fails where there is no GPU
    for written, other in PAIRS:
        n = {**READ, **WRITTEN}[other][1]
        assert call(**{written: at[other]}) == -22, (written, other)
        assert call(**{written: at[other] + 4 * (n - 1)}) == -22, (written, other)
        assert call(**{written: at[other] - 4 * (WRITTEN[written][1] - 1)}) == -22, (written, other)
        assert call(**{written: at[other] + 4 * n}) == -5, (written, other)  # next to each other
        assert call(**{written: at[other] - 4 * WRITTEN[written][1]}) == -5, (written, other)
    assert call(start_pos=at["new_tokens"]) == -5  # read only


@pytest.mark.gpu
def test_the_binding_refuses_overlapping_arrays():
    i32 = lambda *s: torch.ones(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    storage = torch.zeros(64 * pkv.kv_pool_page_bytes(1), dtype=torch.uint8, device="cuda")
    pool = pkv.kv_pool_create(storage, 1)
    good = {name: i32(*SHAPE.get(name, (n,))) for name, (_, n) in {**READ, **WRITTEN}.items()}
    for written, other in PAIRS:
        both = i32(256)
        n, m = WRITTEN[written][1], {**READ, **WRITTEN}[other][1]
        args = {**good, written: both[:n].view(SHAPE.get(written, (n,))),
                other: both[n - 1:n - 1 + m].view(SHAPE.get(other, (m,)))}
        with pytest.raises(pkv.PkvError, match="EINVAL"):
            pkv.paged_tables_build(pool, **args)
        args[other] = both[n:n + m].view(SHAPE.get(other, (m,)))
        pkv.paged_tables_build(pool, **args)
    pool.close()
