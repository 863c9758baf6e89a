"""token_logprobs when a wait gives up: the workspace's error word says so, no row
looks valid that was not worked out, and a reset makes the workspace as new."""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv

ROWS, VOCAB, TOP = 3, 128256, 5


def make(rows=ROWS, vocab=VOCAB, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(torch.bfloat16)
    return x, torch.arange(rows, dtype=torch.int32, device="cuda")


def call(x, targets, ws, top=TOP):
    f = lambda *s: torch.full(s, -77.0, device="cuda")  # noqa: E731
    out = f(len(x)), f(len(x)), torch.full((len(x), top), -77, dtype=torch.int32, device="cuda"), f(len(x), top)
    pkv.token_logprobs(x, targets, *out, ws)
    torch.cuda.synchronize()
    return out


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


def none(out):
    lp, h, ids, tl = out
    return bool(lp.isnan().all() and h.isnan().all() and tl.isnan().all() and (ids == 0).all())


def test_refusals():
    lib, bits = pkv.lib(), pkv._binding._i(0)
    assert lib.token_logprobs_get_error(None, bits, 0) == -22
    assert lib.token_logprobs_get_error(256, None, 0) == -22
    assert lib.token_logprobs_get_error(264, bits, 0) == -22
    with pytest.raises(ValueError, match="CUDA"):
        pkv.token_logprobs_get_error(torch.zeros(1024, dtype=torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,vocab", [(1, 128256), (3, 9000), (64, 40000), (600, 3000), (600, 128256)])
def test_a_wait_that_gives_up(rows, vocab):
    x, targets = make(rows, vocab)
    ws = pkv.alloc_logprobs_workspace(rows, vocab, TOP)
    want = call(x, targets, ws)
    assert pkv.token_logprobs_get_error(ws) == 0
    before = pkv.token_logprobs_set_wait_limit(0)
    try:
        got = call(x, targets, ws)
    finally:
        assert pkv.token_logprobs_set_wait_limit(before) == 0
    assert pkv.token_logprobs_get_error(ws) == pkv.ERR_TIMEOUT
    assert none(got)
    assert none(call(x, targets, ws))  # the workspace is not trusted again
    assert none(call(*make(2, 500, seed=3), ws))
    assert pkv.token_logprobs_get_error(ws, reset=True) == pkv.ERR_TIMEOUT
    assert pkv.token_logprobs_get_error(ws) == 0
    for _ in range(3):
        assert same(call(x, targets, ws), want)


@pytest.mark.gpu
def test_a_short_limit_leaves_values_right_or_nan():
    x, targets = make(700, 6000)
    ws = pkv.alloc_logprobs_workspace(700, 6000, TOP)
    want = call(x, targets, ws)
    before = pkv.token_logprobs_set_wait_limit(1)
    try:
        lp, h, ids, tl = call(x, targets, ws)
    finally:
        pkv.token_logprobs_set_wait_limit(before)
    bits = pkv.token_logprobs_get_error(ws, reset=True)
    lost = lp.isnan()
    assert bits in (0, pkv.ERR_TIMEOUT) and (bits or not lost.any())
    assert torch.equal(lp[~lost], want[0][~lost])
    assert same(call(x, targets, ws), want)


@pytest.mark.gpu
def test_a_reset_clears_what_a_broken_call_left():
    """Counter and tickets that a call did not bring back to zero."""
    x, targets = make()
    ws = pkv.alloc_logprobs_workspace(ROWS, VOCAB, TOP)
    want = call(x, targets, ws)
    words = ws.view(torch.int32)
    words[:64] = 3
    words[0] = pkv.ERR_TIMEOUT
    assert none(call(x, targets, ws))
    assert pkv.token_logprobs_get_error(ws, reset=True) == pkv.ERR_TIMEOUT
    for _ in range(2):
        assert same(call(x, targets, ws), want)


@pytest.mark.gpu
def test_outputs_that_are_left_out_stay_so():
    x, targets = make()
    ws = pkv.alloc_logprobs_workspace(ROWS, VOCAB, TOP)
    ws.view(torch.int32)[0] = pkv.ERR_TIMEOUT
    h = torch.full((ROWS,), -77.0, device="cuda")
    pkv.token_logprobs(x, None, None, h, None, None, ws)
    assert bool(h.isnan().all())
    lp = torch.full((ROWS,), -77.0, device="cuda")
    pkv.token_logprobs(x, targets, lp, None, None, None, ws)
    assert bool(lp.isnan().all())
