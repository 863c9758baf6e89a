"""paged_tables_build against a plain Python walk of the same rule: sequences
in order, each layer's new blocks from the free list, slots by position.
Everything is whole numbers, so results are compared for equality."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

PAGE = 16


def plan(start, new, free, head, tables, num_pages, capacity):
    """The expected outputs, and the error bits."""
    layers, batch, cols = tables.shape
    tables = tables.copy()
    cu, seq_lens, bits = [0], [], 0
    positions = np.zeros(capacity, np.int32)
    slots = np.full((layers, capacity), -1, np.int32)
    room = (len(free) - head) // layers
    asked = taken = 0
    row = 0  # tokens counted so far
    for b in range(batch):
        s, n = int(start[b]), int(new[b])
        ok = s >= 0 and n >= 0 and s + n <= cols * PAGE and row + max(n, 0) <= capacity
        have, want = -(-s // PAGE), -(-(s + n) // PAGE)
        need = want - have if ok else 0
        asked += need
        fits = need == 0 or asked <= room
        if not ok:
            bits |= pkv.ERR_SEQ_LEN
        if not fits:
            bits |= pkv.ERR_NO_PAGES
        served = ok and fits
        if served:
            for layer in range(layers):
                for i in range(need):
                    page = int(free[head + (asked - need) * layers + layer * need + i])
                    if not 0 <= page < num_pages:
                        bits |= pkv.ERR_PAGE_ID
                        page = -1
                    tables[layer, b, have + i] = page
                for t in range(n):
                    page = int(tables[layer, b, (s + t) // PAGE])
                    if not 0 <= page < num_pages:
                        bits |= pkv.ERR_PAGE_ID
                    else:
                        slots[layer, row + t] = page * PAGE + (s + t) % PAGE
            positions[row:row + n] = range(s, s + n)
            taken += need
        row += max(n, 0)
        cu.append(row)
        seq_lens.append(s + n if served else max(s, 0))
    return tables, np.array(cu), np.array(seq_lens), positions, slots, head + taken * layers, bits


def build(start, new, free, head, tables, num_pages, capacity, stream=None):
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    storage = torch.empty(num_pages * pkv.kv_pool_page_bytes(1), dtype=torch.uint8, device="cuda")
    pool = pkv.kv_pool_create(storage, 1)
    batch, layers = len(start), tables.shape[0]
    t = dev(tables)
    outs = dict(cu=dev([-5] * (batch + 1)), lens=dev([-5] * batch), pos=dev([-5] * capacity),
                slots=dev(np.full((layers, capacity), -5)), head=dev([-5]))
    pkv.paged_tables_build(pool, dev(start), dev(new), dev(free), dev([head]), outs["head"], t, outs["cu"],
                           outs["lens"], outs["pos"], outs["slots"], stream=stream)
    bits = pkv.pkv_get_error(pool)
    pool.close()
    c = lambda x: x.cpu().numpy()  # noqa: E731
    return c(t), c(outs["cu"]), c(outs["lens"]), c(outs["pos"]), c(outs["slots"]), int(outs["head"]), bits


def check(start, new, free, head, tables, num_pages, capacity):
    got = build(start, new, free, head, tables, num_pages, capacity)
    want = plan(start, new, free, head, tables, num_pages, capacity)
    for name, a, b in zip(("block_tables", "cu_tokens", "seq_lens", "positions", "slot_map"), got, want):
        assert np.array_equal(a, b), name
    assert got[5:] == want[5:]
    return got


def case(seed, batch, layers, context, cols, chunk, spare=40, free_less=0):
    rng = np.random.default_rng(seed)
    start = rng.integers(0, context + 1, batch)
    new = np.where(rng.random(batch) < 0.3, rng.integers(0, chunk + 1, batch), 1)
    held = -(-start // PAGE)
    need = -(-(start + new) // PAGE) - held
    pages = int((held.sum() + need.sum()) * layers + spare)
    perm = rng.permutation(pages)
    tables = np.full((layers, batch, cols), -1, np.int32)
    at = 0
    for layer in range(layers):
        for b in range(batch):
            tables[layer, b, :held[b]] = perm[at:at + held[b]]
            at += held[b]
    free = perm[at:len(perm) - free_less]
    return start, new, free, int(rng.integers(0, 5)), tables, pages, int(np.maximum(new, 0).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("batch,layers,context,chunk", [
    (1, 1, 0, 1), (1, 3, 31, 40), (2, 16, 16, 17), (64, 16, 300, 1), (255, 2, 90, 33), (256, 2, 64, 20),
    (257, 1, 64, 20), (600, 3, 40, 5)])
@pytest.mark.parametrize("extra", [0, 1, 77])
def test_tables_match_the_rule(batch, layers, context, chunk, extra):
    start, new, free, head, tables, pages, total = case(batch + extra, batch, layers, context,
                                                        (context + chunk) // PAGE + 2, chunk)
    got = check(start, new, free, head, tables, pages, total + extra)
    assert got[6] == 0


@pytest.mark.gpu
def test_largest_batch():
    n = pkv.TABLES_MAX_BATCH
    start = np.arange(n) % 40
    new = 1 + (np.arange(n) % 3)
    need = -(-(start + new) // PAGE) - -(-start // PAGE)
    pages = n * 3 + int(need.sum())
    tables = np.arange(n * 3, dtype=np.int32).reshape(1, n, 3)
    got = check(start, new, np.arange(n * 3, pages), 0, tables, pages, int(new.sum()))
    assert got[6] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("free_less", [1, 30, 60, 10**6])
def test_too_few_pages_serve_the_first_sequences(free_less):
    start, new, free, head, tables, pages, total = case(5, 40, 2, 60, 12, 60, spare=6, free_less=0)
    free = free[:max(len(free) - free_less, head)]
    got = check(start, new, free, head, tables, pages, total + 3)
    need = sum(-(-(s + n) // PAGE) - -(-s // PAGE) for s, n in zip(start, new))
    assert got[6] == (pkv.ERR_NO_PAGES if need > (len(free) - head) // 2 else 0)
    assert got[5] <= len(free)


@pytest.mark.gpu
def test_bad_lengths_pages_and_heads_are_flagged_and_skipped():
    start, new, free, head, tables, pages, total = case(7, 12, 3, 60, 12, 30)
    start[2], new[5] = -3, -1
    start[8], new[8] = 12 * PAGE - 2, 3          # past the block table
    assert check(start, new, free, head, tables, pages, total)[6] == pkv.ERR_SEQ_LEN
    start, new, free, head, tables, pages, total = case(8, 12, 3, 60, 12, 30)
    assert check(start, new, free, head, tables, pages, total - 4)[6] == pkv.ERR_SEQ_LEN  # past the capacity
    free = free.copy()
    free[head], free[head + 3] = pages, -1       # ids outside the pool
    assert check(start, new, free, head, tables, pages, total)[6] == pkv.ERR_PAGE_ID
    start, new, free, head, tables, pages, total = case(9, 6, 2, 60, 12, 30)
    start[1], new[1], tables[1, 1, 2] = 33, 4, -1  # a begun page that the table does not hold
    assert check(start, new, free, head, tables, pages, int(new.sum()))[6] == pkv.ERR_PAGE_ID
    for head in (-1, len(free) + 1):             # a head outside the list: no pages
        start, new, free, _, tables, pages, total = case(9, 6, 2, 60, 12, 30)
        got = build(start, new, free, head, tables, pages, total)
        assert got[6] == pkv.ERR_NO_PAGES and got[5] == head


@pytest.mark.gpu
def test_empty_steps():
    tables = np.full((2, 0, 4), -1, np.int32)
    got = build([], [], [1, 2], 0, tables, 8, 5)
    assert got[1].tolist() == [0] and got[3].tolist() == [0] * 5 and (got[4] == -1).all() and got[5:] == (0, 0)
    tables = np.arange(8, dtype=np.int32).reshape(2, 1, 4)
    got = check([20], [0], [], 0, tables, 8, 0)
    assert got[2].tolist() == [20] and got[6] == 0


@pytest.mark.gpu
def test_another_stream_and_a_graph():
    start, new, free, head, tables, pages, total = case(11, 30, 4, 100, 12, 50)
    side = torch.cuda.Stream()
    want = plan(start, new, free, head, tables, pages, total)
    with torch.cuda.stream(side):
        got = build(start, new, free, head, tables, pages, total)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_refusals():
    """Argument checks of the binding and the library; no CUDA call runs."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool = pkv.KVPool(0, None, 8)
    good = dict(start_pos=i32(4), new_tokens=i32(4), free_pages=i32(9), free_head=i32(1), free_head_out=i32(1),
                block_tables=i32(2, 4, 5), cu_tokens=i32(5), seq_lens=i32(4), positions=i32(7), slot_map=i32(2, 7))
    for name, bad in (("start_pos", i32(3)), ("new_tokens", i32(4, 1)), ("free_head", i32(2)),
                      ("cu_tokens", i32(4)), ("seq_lens", i32(5)), ("slot_map", i32(1, 7)),
                      ("block_tables", i32(4, 5)), ("positions", i32(7, 1))):
        with pytest.raises(ValueError):
            pkv.paged_tables_build(pool, **{**good, name: bad})
    lib = pkv.lib()
    lib_args = [None, 1, 1, 4, 2, 1, 9, 1, 2, 1, 5, 1, 1, 1, 1, 7, None]
    assert lib.paged_tables_build(*lib_args) == -22  # no pool


@pytest.mark.gpu
def test_library_refusals():
    storage = torch.zeros(64 * pkv.kv_pool_page_bytes(1), dtype=torch.uint8, device="cuda")
    pool = pkv.kv_pool_create(storage, 1)
    w = torch.zeros(4096, dtype=torch.int32, device="cuda").data_ptr()
    good = [pool.handle, w, w, 4, 2, w, 9, w, w + 64, w, 5, w, w, w, w, 7, None]
    lib = pkv.lib()
    for i, bad in ((3, -1), (3, pkv.TABLES_MAX_BATCH + 1), (4, 0), (6, -1), (10, 0), (15, -1), (15, 1 << 29),
                   (10, 1 << 27), (1, None), (2, None), (5, None), (7, None), (8, None), (8, w), (9, None),
                   (11, None), (12, None), (13, None), (14, None)):
        args = list(good)
        args[i] = bad
        assert lib.paged_tables_build(*args) == -22, i
    assert ctypes.c_int(lib.pkv_last_cuda_error()).value >= 0
    pool.close()
