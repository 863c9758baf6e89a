"""A cap far above the scores leaves them as they are.

softcap tanh(s / softcap) differs from s by |s|^3 / (3 softcap^2), below 1e-6 for
|s| <= 60 and softcap >= 1e6, so attention with such a cap must agree with
attention without one. Tolerance: the prefill's polynomial is within 2^-17 of
the score, the scores' scaling rounds twice on either side (2^-22 in all), and a
weight of either side is off by 2^-17 + 2^-21 besides, so the weights differ by a
factor 1 + e with e = |s| (2^-17 + 2^-22) + 2 (2^-17 + 2^-21) + 1e-6 and the
outputs by at most 2 e max |v|.
"""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

HQ, HKV, SCALE = 8, 2, 0.125


def setup(lens, max_blocks):
    g = torch.Generator().manual_seed(17)
    pages = sum(-(-n // 16) for n in lens)
    pool = torch.randn(pages, HKV, 2, 16, 64, generator=g).to(torch.bfloat16).cuda()
    tables = torch.full((len(lens), max_blocks), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        tables[b, :-(-n // 16)] = torch.arange(at, at - (-n // 16))
        at -= -n // 16
    return pool, tables.cuda(), g


def agree(plain, capped, q, pool):
    s = float(q.abs().max()) * float(pool[:, :, 0].float().abs().sum(-1).max()) * SCALE
    assert s <= 60
    e = s * (2.0 ** -17 + 2.0 ** -22) + 2 * (2.0 ** -17 + 2.0 ** -21) + 1e-6
    assert float((plain - capped).abs().max()) <= 2 * e * float(pool[:, :, 1].float().abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e6, 1e9, 1e30])
@pytest.mark.parametrize("max_blocks", [40, 2100])  # either decode kernel
def test_decode(softcap, max_blocks):
    lens = [1, 40, 333, 600]
    pool, tables, g = setup(lens, max_blocks)
    handle = pkv.kv_pool_create(pool, HKV)
    q = torch.randn(len(lens), HQ, 64, generator=g).cuda()
    ws = pkv.alloc_decode_workspace(len(lens), HQ, HKV, max_blocks)
    out = [torch.empty(len(lens), HQ, 64, device="cuda") for _ in range(2)]
    for o, cap in zip(out, (0.0, softcap)):
        pkv.paged_gqa_decode_scored(handle, q, o, tables, torch.tensor(lens, dtype=torch.int32, device="cuda"), SCALE,
                                    ws, softcap=cap)
    agree(*out, q, pool)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e6, 1e9, 1e30])
def test_prefill(softcap):
    lens = [1, 40, 333]
    pool, tables, g = setup(lens, 24)
    handle = pkv.kv_pool_create(pool, HKV)
    q = torch.randn(sum(lens), HQ, 64, generator=g).cuda()
    ws = pkv.alloc_prefill_workspace(sum(lens), len(lens), 24)
    cu = torch.tensor([0, 1, 41, 374], dtype=torch.int32, device="cuda")
    out = [torch.empty(sum(lens), HQ, 64, device="cuda") for _ in range(2)]
    for o, cap in zip(out, (0.0, softcap)):
        pkv.paged_gqa_prefill_scored(handle, q, o, tables, cu, torch.zeros(3, dtype=torch.int32, device="cuda"), SCALE,
                                     ws, softcap=cap)
    agree(*out, q, pool)
    handle.close()


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [20.0, 1e6])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_does_not_depend_on_what_was_there(softcap, dtype):
    """Bit for bit the same after a call that left large keys in the memory of the SMs and after one that left zeros."""
    lens = [1, 40, 333, 5, 18]
    pool, tables, g = setup(lens, 24)
    q = (torch.randn(sum(lens), HQ, 64, generator=g) * 0.05).cuda()
    ws = pkv.alloc_prefill_workspace(4096, 12, 24)

    def run(pool, tables, q, chunks, out):
        handle = pkv.kv_pool_create(pool, HKV)
        i32 = dict(dtype=torch.int32, device="cuda")
        cu = torch.tensor([0] + [sum(chunks[:i + 1]) for i in range(len(chunks))], **i32)
        pkv.paged_gqa_prefill_scored(handle, q, out, tables, cu, torch.zeros(len(chunks), **i32), SCALE, ws,
                                     softcap=softcap)
        torch.cuda.synchronize()
        handle.close()
        return out

    outs = []
    for value in (2.0 ** 14, 0.0):
        other = torch.full((24 * 12, HKV, 2, 16, 64), value, dtype=torch.bfloat16, device="cuda")
        t = torch.arange(24 * 12, dtype=torch.int32, device="cuda").view(12, 24)[:, :21].contiguous()
        run(other, t, torch.ones(12 * 330, HQ, 64, device="cuda"), [330] * 12,
            torch.empty(12 * 330, HQ, 64, dtype=dtype, device="cuda"))
        outs.append(run(pool, tables, q, lens, torch.empty(sum(lens), HQ, 64, dtype=dtype, device="cuda")))
    assert torch.equal(*outs)
