"""paged_gqa_decode_scored and paged_gqa_prefill_scored against the formula in
64 bits: capped, distance-biased and windowed scores, documents, prefixes,
rows that see no key; NaN in every slot that no query may read.

Tolerance, per output element. The kernels hold q and the weights p as pairs
of bf16 (each within 2^-17 of its fp32 value: two half steps of 2^-9, doubled),
sum in fp32 and evaluate 2^x and 1/x to about 2^-22. With A the largest
sum_d |q_d k_d| * scale over the row's keys, a score is off by at most
A (2^-17 + 64 * 2^-24) + |score| 2^-23, capping and its bias add at most
softcap * 2^-20 and |bias| * 2^-22 (tanh has slope at most 1), so a weight is
off by a factor 1 + e with e = that sum + 2^-17 + 2^-21, and the output by at
most 2 e sum p |v| / sum p. Rounding to the output type adds half a step; where the
output is bf16 the prefill also rounds its weights to bf16, a factor within
1 + 2^-8 each, so e grows by 2^-8.
"""
import numpy as np
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

D, PAGE = 64, 16
SCALE = 0.125


def reference(q, k, v, pos, lo, hi, softcap, slopes, weight_error=0.0):
    """One sequence: q [N,Hq,64], k/v [keys,Hkv,64] fp64, row n at position
    pos[n] sees keys lo[n] <= j < hi[n]. Returns out and its tolerance."""
    n, hq = q.shape[:2]
    group = hq // k.shape[1]
    out, tol = np.zeros((n, hq, D)), np.zeros((n, hq, D))
    for i in range(n):
        if hi[i] <= lo[i]:
            continue
        j = np.arange(lo[i], hi[i])
        for h in range(hq):
            kk, vv = k[j, h // group], v[j, h // group]
            s = SCALE * (kk @ q[i, h])
            size = SCALE * (np.abs(kk) @ np.abs(q[i, h])).max()
            e = weight_error + size * (2.0 ** -17 + 64 * 2.0 ** -24 + 2.0 ** -23) + 2.0 ** -17 + 2.0 ** -21
            if softcap:
                s = softcap * np.tanh(s / softcap)
                e += softcap * 2.0 ** -20
            if slopes is not None:
                bias = slopes[h] * np.abs(pos[i] - j)
                s = s - bias
                # keys whose weight is 0 in fp32 carry no error: only biases within 110 of the smallest count
                near = np.abs(bias)[s > s.max() - 110.0]
                e += near.max() * 2.0 ** -22
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vv
            tol[i, h] = 2 * e * (p @ np.abs(vv))
    return out, tol


def spread(rng, counts, max_blocks, hkv, spare=5):
    """Scattered pages for page ranges [(first, last)) per sequence, everything NaN."""
    total = sum(b - a for a, b in counts)
    perm = rng.permutation(total + spare)
    tables = np.full((len(counts), max_blocks), -1, np.int64)
    at = 0
    for b, (x, y) in enumerate(counts):
        tables[b, :x] = -7 - b  # given back: must not be looked up
        tables[b, x:y] = perm[at:at + y - x]
        at += y - x
    pool = torch.full((total + spare, hkv, 2, PAGE, D), float("nan"), dtype=torch.bfloat16)
    return tables, pool


def fill(rng, pool, tables, b, lo, hi):
    """Random K and V at positions [lo, hi) of sequence b; fp64 copies [hi, Hkv, 64]."""
    hkv = pool.shape[1]
    kv = torch.from_numpy(rng.standard_normal((2, max(hi, 0), hkv, D))).to(torch.bfloat16)
    kv[0, rng.integers(0, max(hi, 1), 2 if hi else 0)] *= 4
    for t in range(lo, hi):
        pool[tables[b, t // PAGE], :, 0, t % PAGE] = kv[0, t]
        pool[tables[b, t // PAGE], :, 1, t % PAGE] = kv[1, t]
    kv = kv.double().numpy()
    return kv[0], kv[1]


def compare(got, want, tol, dtype):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    got = got.double().cpu().numpy()
    limit = tol + half * (np.abs(want) + tol) + 1e-38
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / limit).max() if got.size else 0.0
    assert worst <= 1.0, f"worst error {worst:.3g} of the tolerance"


def run_decode(seed, hq, hkv, lens, softcap=0.0, alibi=False, window=0, first=None, dtype=torch.float32,
               max_blocks=None, stream=None):
    rng = np.random.default_rng(seed)
    lo = [max(n - window if window else 0, first[b] if first else 0, 0) for b, n in enumerate(lens)]
    max_blocks = max_blocks or max(-(-max(n, 1) // PAGE) for n in lens) + 2
    ranges = [(min(a, n) // PAGE if a < n else 0, -(-n // PAGE) if a < n else 0) for a, n in zip(lo, lens)]
    tables, pool = spread(rng, ranges, max_blocks, hkv)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, D)) * 2).float()
    slopes = (2.0 ** (-8.0 * (1 + np.arange(hq)) / hq)).astype(np.float32) if alibi else None
    want, tol = np.zeros((len(lens), hq, D)), np.zeros((len(lens), hq, D))
    for b, n in enumerate(lens):
        if lo[b] >= n:
            continue
        k, v = fill(rng, pool, tables, b, lo[b], n)
        o, t = reference(q[b:b + 1].double().numpy(), k, v, [n - 1], [lo[b]], [n], softcap, slopes)
        want[b], tol[b] = o[0], t[0]
    storage = pool.cuda()
    handle = pkv.kv_pool_create(storage, hkv)
    out = torch.full((len(lens), hq, D), float("nan"), dtype=dtype, device="cuda")
    ws = pkv.alloc_decode_workspace(len(lens), hq, hkv, max_blocks)
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
    kw = dict(softcap=softcap, alibi_slopes=torch.from_numpy(slopes).cuda() if alibi else None, window=window,
              first_keys=i32(first) if first else None)
    q, tables, lens = q.cuda(), i32(tables), i32(lens)
    for _ in range(2):  # the workspace is left ready
        pkv.paged_gqa_decode_scored(handle, q, out, tables, lens, SCALE, ws, stream=stream, **kw)
    assert pkv.pkv_get_error(handle) == 0
    compare(out, want, tol, dtype)
    handle.close()


LENS = [1, 2, 15, 16, 17, 33, 160, 700]

# Block tables that could hold long sequences (2100 pages) take the general
# kernel, narrow ones the kernel for little work.
WIDE = pytest.mark.parametrize("max_blocks", [None, 2100], ids=["narrow", "wide"])


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(32, 8), (14, 2), (3, 3), (8, 1), (15, 5), (6, 3), (10, 2), (12, 2)])
@pytest.mark.parametrize("softcap,alibi,window", [(0.0, False, 0), (20.0, False, 0), (0.0, True, 0), (5.0, True, 40)])
@WIDE
def test_decode_groups_and_scores(hq, hkv, softcap, alibi, window, max_blocks):
    run_decode(hq + window, hq, hkv, LENS, softcap, alibi, window, max_blocks=max_blocks)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 100, 699, 700, 5000, 2**31 - 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@WIDE
def test_decode_windows(window, dtype, max_blocks):
    # (a window bounds the pages that count: many sequences take the general kernel with it)
    run_decode(window % 1000, 8, 2, LENS * (1 if max_blocks is None else 60), 30.0, True, window, dtype=dtype,
               max_blocks=max_blocks)


@pytest.mark.gpu
@WIDE
def test_decode_first_keys_and_rows_that_see_nothing(max_blocks):
    run_decode(1, 8, 4, LENS, 0.0, False, 0, first=[0, -5, 3, 16, 16, 32, 100, 2**31 - 1], max_blocks=max_blocks)
    run_decode(2, 8, 4, LENS, 10.0, True, 0, first=[1, 5, 14, 15, 0, 31, 1000, 690], dtype=torch.bfloat16,
               max_blocks=max_blocks)
    run_decode(2, 8, 4, LENS, 10.0, True, 20, first=[1, 5, 14, 15, 0, 31, 1000, 690], dtype=torch.bfloat16)
    run_decode(3, 8, 4, [9, 40], first=[9, 40], max_blocks=max_blocks)  # all rows empty


@pytest.mark.gpu
def test_decode_one_long_sequence_and_many_short_ones():
    run_decode(4, 32, 8, [9000], 50.0, False, 0)
    run_decode(5, 14, 2, [20000, 3], 0.0, True, 0, dtype=torch.bfloat16)
    run_decode(6, 4, 2, [1 + (7 * i) % 37 for i in range(1100)], 50.0, False, 8)
    run_decode(6, 4, 2, [1 + (7 * i) % 37 for i in range(1100)], 50.0, True, 0, max_blocks=1100)  # two launches


@pytest.mark.gpu
def test_decode_without_scoring_is_the_plain_decode():
    rng = np.random.default_rng(7)
    lens = [5, 300, 1200]
    tables, pool = spread(rng, [(0, -(-n // PAGE)) for n in lens], 80, 8)
    kv = [fill(rng, pool, tables, b, 0, n) for b, n in enumerate(lens)]
    handle = pkv.kv_pool_create(pool.cuda(), 8)
    q = torch.from_numpy(rng.standard_normal((3, 32, D))).float().cuda()
    ws = pkv.alloc_decode_workspace(3, 32, 8, 80)
    a, b = torch.empty_like(q), torch.empty_like(q)
    tables = torch.tensor(tables, dtype=torch.int32, device="cuda")
    dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pkv.paged_gqa_decode(handle, q, a, tables, dev_lens, SCALE, ws)
    pkv.paged_gqa_decode_scored(handle, q, b, tables, dev_lens, SCALE, ws)
    assert pkv.pkv_get_error(handle) == 0
    # (not the same bits: few sequences take a kernel of their own)
    for i, n in enumerate(lens):
        want, tol = reference(q[i:i + 1].double().cpu().numpy(), *kv[i], [n - 1], [0], [n], 0.0, None)
        compare(a[i:i + 1], want, tol, torch.float32)
        compare(b[i:i + 1], want, tol, torch.float32)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("max_blocks", [4, 2100], ids=["narrow", "wide"])
def test_decode_bad_lengths_and_pages(max_blocks):
    rng = np.random.default_rng(8)
    lens = [40, 0, -3, 16 * max_blocks + 1, 20]
    tables, pool = spread(rng, [(0, 3), (0, 0), (0, 0), (0, 0), (0, 2)], max_blocks, 2)
    k, v = fill(rng, pool, tables, 0, 0, 40)
    k4, v4 = fill(rng, pool, tables, 4, 0, 20)
    tables[0, 1] = 10**6  # a bad page: its keys are skipped
    handle = pkv.kv_pool_create(pool.cuda(), 2)
    q = torch.from_numpy(rng.standard_normal((5, 8, D))).float()
    out = torch.full((5, 8, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.paged_gqa_decode_scored(handle, q.cuda(), out, i32(tables), i32(lens), SCALE,
                                pkv.alloc_decode_workspace(5, 8, 2, max_blocks), softcap=9.0)
    assert pkv.pkv_get_error(handle) == pkv.ERR_SEQ_LEN | pkv.ERR_PAGE_ID
    assert (out[1:4] == 0).all()
    keep = np.r_[0:16, 32:40]
    o, t = reference(q[:1].double().numpy(), k[keep], v[keep], [39], [0], [24], 9.0, None)
    compare(out[:1], o, t, torch.bfloat16)
    o, t = reference(q[4:].double().numpy(), k4, v4, [19], [0], [20], 9.0, None)
    compare(out[4:], o, t, torch.bfloat16)
    handle.close()


def run_prefill(seed, hq, hkv, chunks, starts, softcap=0.0, alibi=False, window=0, docs=None, prefix=None,
                dtype=torch.float32, check=None):
    """docs: per sequence a function position -> first visible position."""
    rng = np.random.default_rng(seed)
    total = sum(chunks)
    lens = [a + b for a, b in zip(chunks, starts)]
    max_blocks = -(-max(lens) // PAGE) + 1
    rows = []  # (pos, lo, hi) per sequence
    doc_starts = np.zeros(total, np.int64)
    at = 0
    for b, (n, s) in enumerate(zip(chunks, starts)):
        pos = np.arange(s, s + n)
        doc = np.array([docs(b, int(i)) for i in pos], np.int64) if docs else np.zeros(n, np.int64)
        doc_starts[at:at + n] = doc
        lo = np.maximum(doc, pos - window + 1 if window else 0).clip(0)
        hi = np.maximum(pos + 1, min(prefix[b], s + n) if prefix else 0)
        rows.append((pos, lo, hi))
        at += n
    seen = [(min([x for x, y in zip(lo, hi) if x < y], default=0), max([y for x, y in zip(lo, hi) if x < y], default=0))
            for _, lo, hi in rows]
    tables, pool = spread(rng, [(a // PAGE, -(-b // PAGE)) for a, b in seen], max_blocks, hkv)
    q = torch.from_numpy(rng.standard_normal((total, hq, D)) * 2).float()
    slopes = (2.0 ** (-8.0 * (1 + np.arange(hq)) / hq)).astype(np.float32) if alibi else None
    want, tol, at = np.zeros((total, hq, D)), np.zeros((total, hq, D)), 0
    for b, (pos, lo, hi) in enumerate(rows):
        k, v = fill(rng, pool, tables, b, *seen[b])
        n = len(pos)
        want[at:at + n], tol[at:at + n] = reference(q[at:at + n].double().numpy(), k, v, pos, lo, hi, softcap, slopes,
                                                  2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
        at += n
    handle = pkv.kv_pool_create(pool.cuda(), hkv)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((total, hq, D), float("nan"), dtype=dtype, device="cuda")
    pkv.paged_gqa_prefill_scored(handle, q.cuda(), out, i32(tables), i32(np.r_[0, np.cumsum(chunks)]), i32(starts),
                                 SCALE, pkv.alloc_prefill_workspace(total, len(chunks), max_blocks), softcap=softcap,
                                 alibi_slopes=torch.from_numpy(slopes).cuda() if alibi else None, window=window,
                                 prefix_lens=i32(prefix) if prefix else None,
                                 doc_starts=i32(doc_starts) if docs else None)
    assert pkv.pkv_get_error(handle) == 0
    compare(out, want, tol, dtype)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(8, 2), (7, 1), (2, 2), (8, 1), (6, 2), (10, 5), (5, 1), (6, 1)])
@pytest.mark.parametrize("softcap,alibi,window", [(0.0, False, 0), (20.0, False, 0), (0.0, True, 0), (5.0, True, 40)])
def test_prefill_groups_and_scores(hq, hkv, softcap, alibi, window):
    run_prefill(hq + window, hq, hkv, [1, 70, 33], [0, 5, 130], softcap, alibi, window)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 16, 17, 63, 64, 65, 129, 2**31 - 1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_windows(window, dtype):
    run_prefill(window % 1000, 4, 1, [200, 3, 64], [0, 333, 64], 30.0, True, window, dtype=dtype)


@pytest.mark.gpu
def test_prefill_documents():
    for size in (1, 5, 16, 50, 64, 100, 1000):
        run_prefill(size, 4, 2, [150, 40], [0, 77], 0.0, True, 0, docs=lambda b, i: i // size * size)
    run_prefill(9, 4, 2, [150, 40], [0, 77], 12.0, False, 30, docs=lambda b, i: i // 50 * 50, dtype=torch.bfloat16)


@pytest.mark.gpu
def test_prefill_prefixes():
    run_prefill(10, 4, 2, [100, 40, 7], [0, 77, 0], 0.0, True, 0, prefix=[30, 100, 0])
    run_prefill(11, 4, 2, [100, 40, 7], [0, 77, 0], 20.0, False, 0, prefix=[2**31 - 1, 10, 7])
    run_prefill(12, 4, 2, [150, 40], [0, 77], 0.0, False, 25, prefix=[90, 200], dtype=torch.bfloat16)
    run_prefill(13, 7, 1, [150, 70], [0, 300], 0.0, True, 0, prefix=[128, 364], docs=lambda b, i: 0 if i < 40 else 40)


@pytest.mark.gpu
def test_prefill_rows_that_see_nothing():
    # documents that start after the token, here and there and everywhere
    run_prefill(14, 4, 2, [90, 40], [0, 77], docs=lambda b, i: 10**6 if i % 3 == 0 else 0)
    run_prefill(15, 4, 2, [90, 40], [0, 77], 8.0, True, docs=lambda b, i: 10**6 if b == 0 else i)
    run_prefill(16, 4, 2, [20, 3], [0, 7], docs=lambda b, i: 10**6)
    run_prefill(17, 4, 2, [200], [100], docs=lambda b, i: 180 if i < 180 else i, prefix=[256])


@pytest.mark.gpu
def test_prefill_long_chunks():
    run_prefill(18, 4, 1, [600], [1500], 50.0, False, 700)
    run_prefill(19, 2, 2, [1000, 1], [0, 2000], 0.0, True, 0, dtype=torch.bfloat16)


@pytest.mark.gpu
def test_prefill_without_scoring_is_the_plain_prefill():
    """The same rows as paged_prefill's attention, from the queries and pages it leaves."""
    rng = np.random.default_rng(20)
    chunks, hq, hkv = [130, 55], 8, 2
    total = sum(chunks)
    q, k, v = (torch.from_numpy(rng.standard_normal((total, h, D))).to(torch.bfloat16).cuda() for h in (hq, hkv, hkv))
    storage = torch.zeros(40, hkv, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    handle = pkv.kv_pool_create(storage, hkv)
    tables = torch.from_numpy(rng.permutation(40)[:28].astype(np.int32).reshape(2, 14)).cuda()
    cu = torch.tensor([0, 130, 185], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = pkv.alloc_prefill_workspace(total, 2, 14)
    q_rot, a, b = (torch.empty(total, hq, D, device="cuda") for _ in range(3))
    pkv.paged_prefill(handle, q, k, v, q_rot, a, tables, cu, start, pkv.build_rope_table(10000.0, 224), SCALE, ws)
    pkv.paged_gqa_prefill_scored(handle, q_rot, b, tables, cu, start, SCALE, ws)
    assert pkv.pkv_get_error(handle) == 0
    # (not the same bits: the two take a row's keys in opposite orders)
    at = 0
    for s, n in enumerate(chunks):
        pages = storage[tables[s].long()].double().cpu().numpy()  # [14, Hkv, 2, 16, 64]
        kv = pages.transpose(2, 1, 0, 3, 4).reshape(2, hkv, -1, D).transpose(0, 2, 1, 3)
        pos = np.arange(n)
        want, tol = reference(q_rot[at:at + n].double().cpu().numpy(), kv[0], kv[1], pos, 0 * pos, pos + 1, 0.0, None)
        compare(a[at:at + n], want, tol, torch.float32)
        compare(b[at:at + n], want, tol, torch.float32)
        at += n
    handle.close()


@pytest.mark.gpu
def test_prefill_bad_starts_ends_and_pages():
    rng = np.random.default_rng(21)
    chunks, starts, hq, hkv = [40, 30, 50], [0, -3, 100], 4, 2
    tables, pool = spread(rng, [(0, 3), (0, 0), (0, 8)], 8, hkv)
    k, v = fill(rng, pool, tables, 0, 0, 40)
    k2, v2 = fill(rng, pool, tables, 2, 0, 128)
    tables[0, 1] = -1
    handle = pkv.kv_pool_create(pool.cuda(), hkv)
    q = torch.from_numpy(rng.standard_normal((120, hq, D))).float()
    out = torch.full((120, hq, D), float("nan"), device="cuda")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    pkv.paged_gqa_prefill_scored(handle, q.cuda(), out, i32(tables), i32([0, 40, 70, 120]), i32(starts), SCALE,
                                 pkv.alloc_prefill_workspace(120, 3, 8), window=64)
    assert pkv.pkv_get_error(handle) == pkv.ERR_SEQ_LEN | pkv.ERR_PAGE_ID
    assert (out[40:70] == 0).all() and (out[98:] == 0).all()  # a negative start; past the block table
    keep = np.r_[0:16, 32:40]
    for t in range(40):
        j = keep[(keep <= t)]
        o, e = reference(q[t:t + 1].double().numpy(), k[j], v[j], [t], [0], [len(j)], 0.0, None)
        compare(out[t:t + 1], o, e, torch.float32)
    pos = np.arange(100, 128)
    o, e = reference(q[70:98].double().numpy(), k2, v2, pos, pos - 63, pos + 1, 0.0, None)
    compare(out[70:98], o, e, torch.float32)
    handle.close()


@pytest.mark.gpu
def test_another_stream_and_a_graph():
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run_decode(22, 8, 2, LENS, 30.0, True, 50)
        run_prefill(23, 8, 2, [1, 70, 33], [0, 5, 130], 30.0, True, 50)


def test_refusals():
    pool = pkv.KVPool(0, None, 8)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    good = dict(q_rot=f(4, 32, 64), out=f(4, 32, 64), block_tables=i32(4, 5), seq_lens=i32(4), scale=0.125,
                workspace=torch.zeros(1024, dtype=torch.uint8))
    for name, bad in (("q_rot", f(4, 32, 32)), ("out", f(4, 31, 64)), ("out", f(4, 32, 64).half()),
                      ("block_tables", i32(3, 5)), ("seq_lens", i32(5))):
        with pytest.raises(ValueError):
            pkv.paged_gqa_decode_scored(pool, **{**good, name: bad})
    with pytest.raises(TypeError):
        pkv.paged_gqa_decode_scored(pool, **{**good, "out": None})
    good = dict(q_rot=f(10, 32, 64), out=f(10, 32, 64), block_tables=i32(2, 5), cu_tokens=i32(3), start_pos=i32(2),
                scale=0.125, workspace=torch.zeros(1024, dtype=torch.uint8))
    for name, bad in (("q_rot", f(10, 32, 32)), ("out", f(9, 32, 64)), ("cu_tokens", i32(2)), ("start_pos", i32(3)),
                      ("block_tables", i32(10))):
        with pytest.raises(ValueError):
            pkv.paged_gqa_prefill_scored(pool, **{**good, name: bad})
    lib = pkv.lib()
    assert lib.paged_gqa_decode_scored(None, 256, 256, 1, 256, 4, 256, None, 2, 32, None, 256, 1 << 20, None) == -22
    assert lib.paged_gqa_prefill_scored(None, 256, 256, 1, 256, 4, 256, 256, None, None, 2, 8, 32, None, 256, 1 << 20,
                                        None) == -22


@pytest.mark.gpu
def test_library_refusals():
    import ctypes

    from paged_kv_decode_rope_gb300._binding import _Scoring
    handle = pkv.kv_pool_create(torch.zeros(8, 2, 2, PAGE, D, dtype=torch.bfloat16, device="cuda"), 2)
    lib, nan, inf = pkv.lib(), float("nan"), float("inf")
    ws = pkv.alloc_decode_workspace(4, 8, 2, 8)
    w, n = ws.data_ptr(), ws.numel()
    sc = lambda *a: ctypes.addressof(keep.append(_Scoring(*a)) or keep[-1])  # noqa: E731
    keep = []
    ok = sc(0.125, 0.0, None, 0)
    good = [handle.handle, w, w, 1, w, 8, w, None, 4, 8, ok, w, n, None]
    bad_scorings = [None, sc(nan, 0.0, None, 0), sc(0.1, -1.0, None, 0), sc(0.1, inf, None, 0), sc(0.1, nan, None, 0),
                    sc(1.0, 1e-39, None, 0), sc(0.1, 0.0, None, -1)]
    for i, values in ((1, [None, w + 4]), (2, [None, w + 8]), (3, [2, -1]), (4, [None]), (5, [0, 1 << 24]),
                      (6, [None]), (8, [-1]), (9, [0, 7, 18]), (10, bad_scorings), (11, [None, w + 16]), (12, [16])):
        for bad in values:
            args = list(good)
            args[i] = bad
            assert lib.paged_gqa_decode_scored(*args) == -22, (i, bad)
    need = pkv.paged_prefill_workspace_bytes(20, 2, 8)
    good = [handle.handle, w, w, 0, w, 8, w, w, None, None, 2, 20, 8, ok, w, need, None]
    for i, values in ((1, [None, w + 4]), (2, [None, w + 8]), (3, [2]), (4, [None]), (5, [0]), (6, [None]), (7, [None]),
                      (10, [-1, 0]), (11, [-1]), (12, [0, 7, 18]), (13, bad_scorings), (14, [None, w + 16]),
                      (15, [need - 1])):
        for bad in values:
            args = list(good)
            args[i] = bad
            assert lib.paged_gqa_prefill_scored(*args) == -22, (i, bad)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("chunks,starts", [([16, 0], [0, 0]), ([0, 16], [0, 270]), ([132, 1, 1], [1, 0, 1])])
def test_prefill_keys_past_the_last_one_seen_may_hold_anything(chunks, starts, dtype):
    # every third token sees nothing, the last of some tiles among them: its own key is NaN
    run_prefill(47, 8, 4, chunks, starts, softcap=20.0, docs=lambda b, p: p // 5 * 5 + (1000 if p % 3 == 0 else 0),
                dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_decode_of_many_windowed_sequences(dtype):
    # enough pages for the general kernel although each sequence sees at most three (and two launches)
    lens = [1 + (7 * i) % 90 for i in range(1100)]
    run_decode(61, 16, 8, lens, 30.0, True, 30, first=[max(0, n - 1 - (5 * i) % 50) for i, n in enumerate(lens)],
               dtype=dtype)
