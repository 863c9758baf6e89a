"""Caps that the folded query scale cannot carry are refused, those at the ends of the
range leave right scores.

A query times 2 log2(e) scale / softcap enters the products as a bf16 pair; past
the range its lower part, or all of it, leaves bf16's exponents. At the upper end
the outputs are those without a cap (|s|^3 / (3 softcap^2) is nothing), within the
2^-17 of the pairs on either side: weights off by a factor 1 + e, e = |s| 2^-16 +
2^-15, outputs by 2 e max |v|. At the lower end every score is +-softcap, a
difference of nothing: the outputs are the means of the values, off by the same
with |s| = 0.
"""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

HQ, HKV, N = 8, 2, 40


def attend(softcap, scale, prefill, pool, q, max_blocks=5):
    handle = pkv.kv_pool_create(pool, HKV)
    i32 = dict(dtype=torch.int32, device="cuda")
    tables = torch.full((1, max_blocks), -1, **i32)
    tables[0, :3] = torch.arange(3, **i32)
    out = torch.full((1, HQ, 64), -77.0, device="cuda")
    try:
        if prefill:
            pkv.paged_gqa_prefill_scored(handle, q, out, tables, torch.tensor([0, 1], **i32),
                                         torch.tensor([N - 1], **i32), scale, pkv.alloc_prefill_workspace(1, 1, max_blocks),
                                         softcap=softcap)
        else:
            pkv.paged_gqa_decode_scored(handle, q, out, tables, torch.tensor([N], **i32), scale,
                                        pkv.alloc_decode_workspace(1, HQ, HKV, max_blocks), softcap=softcap)
        torch.cuda.synchronize()
    finally:
        handle.close()
    return out


def data():
    g = torch.Generator().manual_seed(5)
    return (torch.randn(3, HKV, 2, 16, 64, generator=g).to(torch.bfloat16).cuda(),
            torch.randn(1, HQ, 64, generator=g).cuda())


WAYS = pytest.mark.parametrize("prefill,max_blocks", [(False, 5), (False, 2100), (True, 5)])


@pytest.mark.gpu
@WAYS
@pytest.mark.parametrize("scale,softcap", [(0.125, 2e30), (0.125, 1e38), (0.125, 1e-22), (0.0, 1e33), (-1.0, 9e-21),
                                           (1e25, 100.0)])
def test_caps_out_of_range_are_refused(prefill, max_blocks, scale, softcap):
    with pytest.raises(pkv.PkvError, match="EINVAL"):
        attend(softcap, scale, prefill, *data(), max_blocks)


@pytest.mark.gpu
@WAYS
def test_the_ends_of_the_range(prefill, max_blocks):
    pool, q = data()
    plain = attend(0.0, 0.125, prefill, pool, q, max_blocks)
    s = float(q.abs().max()) * float(pool[:, :, 0].float().abs().sum(-1).max()) * 0.125
    v = pool[:, :, 1].float()
    e = s * 2.0 ** -16 + 2.0 ** -15
    assert float((attend(1e30, 0.125, prefill, pool, q, max_blocks) - plain).abs().max()) <= 2 * e * float(v.abs().max())
    mean = v.permute(1, 0, 2, 3).flatten(1, 2)[:, :N].mean(1).repeat_interleave(HQ // HKV, 0)
    low = attend(2e-21, 0.125, prefill, pool, q, max_blocks)
    assert float((low[0] - mean).abs().max()) <= 2 * 2.0 ** -15 * float(v.abs().max())
