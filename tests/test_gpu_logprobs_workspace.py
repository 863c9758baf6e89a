"""One workspace of token_logprobs serves calls of any row counts in any order.

Expected values are the formulas in 64 bits; the tolerances are those of a sum
of V terms in fp32: |logp| 2^-22 + 2^-20 + V 2^-34 (every term within 2^-21, the
sum within (V / 1024 + 40) 2^-24 of itself, its logarithm rounded once).
"""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

UNWRITTEN = -77.0


def outputs(rows, top):
    f = lambda *s: torch.full(s, UNWRITTEN, device="cuda")  # noqa: E731
    return f(rows), f(rows), torch.full((rows, top), int(UNWRITTEN), dtype=torch.int32, device="cuda"), f(rows, top)


def logits(seed, rows, vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)


def check(x, top, ws):
    rows, vocab = x.shape
    targets = (torch.arange(rows, device="cuda") * 7919 % vocab).to(torch.int32)
    lp, h, ids, tl = outputs(rows, top)
    pkv.token_logprobs(x, targets, lp, h, ids, tl, ws)
    logp = torch.log_softmax(x.double(), dim=-1)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(ids.long(), order), "top_ids"
    base = 2.0 ** -20 + vocab * 2.0 ** -34
    for got, want in ((lp, logp.gather(1, targets.long()[:, None])[:, 0]), (tl, logp.gather(1, order))):
        assert bool(((got.double() - want).abs() <= want.abs() * 2.0 ** -22 + base).all())
    want = torch.special.entr(logp.exp()).sum(-1)
    assert bool(((h.double() - want).abs() <= (want + 1) * (want * 2.0 ** -22 + base)).all()), "entropy"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [(1, 64, 100, 140), (64, 128, 2, 227), (300, 1, 455, 64)])
def test_row_counts_in_any_order(dtype, counts):
    vocab, top = 40000, 5
    ws = pkv.alloc_logprobs_workspace(max(counts), vocab, top)
    for rows in counts:
        check(logits(rows, rows, vocab, dtype), top, ws)
