"""The scores behind an fp32 output have no error of one direction.

Every row sees two keys of scores s and -s with values 1 and -1, so its output is
tanh(s') for the capped score s', and atanh of the output gives s' back.
Tolerance: q enters as a bf16 pair (2^-17 of the score), the two weights as
well (2^-17 of each, so 2^-17 of s' in absolute terms, at most 2^-16 s' for s' >=
0.5), and fp32 roundings add less than 2^-19: one row is within e = 3 * 2^-17 +
2^-19 of s'. Roundings to nearest have no direction: the mean of n rows' errors,
each at most e, is within 6 e / sqrt(n) (six standard deviations).
"""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

HQ, HKV, ROWS, SCALE = 8, 2, 2048, 0.125


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 8.0, 50.0, 1e6])
def test_prefill(softcap):
    g = torch.Generator().manual_seed(23)
    pages = ROWS // 16
    sign = 1.0 - 2.0 * (torch.arange(ROWS) % 2)
    pool = torch.zeros(pages, HKV, 2, 16, 64)
    pool[:, :, 0, :, 0] = sign.view(pages, 1, 16)
    pool[:, :, 1] = sign.view(pages, 1, 16, 1)
    pool = pool.to(torch.bfloat16).cuda()
    q = torch.zeros(ROWS, HQ, 64)
    q[:, :, 0] = 4.0 + 4.0 * torch.rand(ROWS, HQ, generator=g)
    s = SCALE * q[:, :, 0].double()  # 0.5 .. 1
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.empty(ROWS, HQ, 64, device="cuda")
    handle = pkv.kv_pool_create(pool, HKV)
    pkv.paged_gqa_prefill_scored(handle, q.cuda(), out, torch.arange(pages, **i32).view(1, pages),
                                 torch.tensor([0, ROWS], **i32), torch.zeros(1, **i32), SCALE,
                                 pkv.alloc_prefill_workspace(ROWS, 1, pages), softcap=softcap, window=2)
    want = softcap * torch.tanh(s / softcap) if softcap else s
    got = torch.atanh(out.cpu().double()[1:, :, 0])  # the key of value 1 has score s, whichever of the two it is
    off = got / want[1:] - 1.0
    e = 3 * 2.0 ** -17 + 2.0 ** -19
    assert float(off.abs().max()) <= e
    assert abs(float(off.mean())) <= 6 * e / off.numel() ** 0.5
    handle.close()
