"""A key that is not a number, where a query sees it, makes that query's row
NaN, as a softmax over it is; no other sequence or kv head is touched."""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

HQ, HKV, LENS = 8, 2, [40, 700, 1, 333]


def setup(max_blocks, seq, pos):
    g = torch.Generator().manual_seed(23)
    counts = [-(-n // 16) for n in LENS]
    pool = torch.randn(sum(counts), HKV, 2, 16, 64, generator=g).to(torch.bfloat16)
    tables, at = torch.full((len(LENS), max_blocks), -1, dtype=torch.int32), 0
    for b, c in enumerate(counts):
        tables[b, :c] = torch.arange(at, at + c)
        at += c
    for p in pos:
        pool[tables[seq, p // 16], 1, 0, p % 16, 7] = float("nan")  # kv head 1
    return pool.cuda(), tables.cuda(), g


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("max_blocks", [48, 2100])  # either decode kernel
@pytest.mark.parametrize("seq,pos", [(1, [5]), (1, [699]), (1, range(700)), (0, range(16)), (2, [0]), (3, [332])])
def test_decode(seq, pos, max_blocks, softcap):
    pool, tables, g = setup(max_blocks, seq, pos)
    handle = pkv.kv_pool_create(pool, HKV)
    q = torch.randn(len(LENS), HQ, 64, generator=g).cuda()
    out = torch.empty(len(LENS), HQ, 64, device="cuda")
    pkv.paged_gqa_decode_scored(handle, q, out, tables, torch.tensor(LENS, dtype=torch.int32, device="cuda"), 0.125,
                                pkv.alloc_decode_workspace(len(LENS), HQ, HKV, max_blocks), softcap=softcap)
    want = torch.zeros(len(LENS), HQ, dtype=torch.bool)
    want[seq, HQ // HKV:] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), want) and torch.equal(torch.isnan(out).any(-1).cpu(), want)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill(softcap, dtype):
    seq, pos = 1, 310
    pool, tables, g = setup(48, seq, [pos])
    handle = pkv.kv_pool_create(pool, HKV)
    cu = torch.tensor([0, 40, 740, 741, 1074], dtype=torch.int32, device="cuda")
    q = torch.randn(1074, HQ, 64, generator=g).cuda()
    out = torch.empty(1074, HQ, 64, dtype=dtype, device="cuda")
    pkv.paged_gqa_prefill_scored(handle, q, out, tables, cu, torch.zeros(4, dtype=torch.int32, device="cuda"), 0.125,
                                 pkv.alloc_prefill_workspace(1074, 4, 48), softcap=softcap)
    nan = torch.isnan(out).cpu()
    first = 40 + pos  # the first row that sees the key
    assert nan[first:740, HQ // HKV:].all()
    assert not nan[:, :HQ // HKV].any()  # the other kv head
    assert not nan[:40].any() and not nan[740:].any()  # the other sequences
    assert not nan[40:first, HQ // HKV:].any()  # a key whose score is masked
    handle.close()
