"""token_logprobs against the formulas in 64 bits, and the alternatives against
a full sort (largest logit first, the lower id first among equals).

Tolerances. y - m is one rounded product of an exact difference, e^(y-m) is
within 2^-21 of its value (2^x to 2^-22, its argument rounded once), the
sum of V of them adds at most (V / 1024 + 40) roundings of 2^-24 of itself, its
logarithm one of 2^-23: logprobs are within |logp| * 2^-22 + 2^-20 + V 2^-34,
entropies within (H + 1) times the same.
"""
import numpy as np
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv


def expected(x, targets, top, scale):
    """x fp64 [R,V] (numpy)."""
    with np.errstate(all="ignore"):
        y = x * scale
        m = y.max(axis=1, keepdims=True)
        log_s = np.log(np.exp(y - m).sum(axis=1, keepdims=True))
        logp = (y - m) - log_s  # y - (m + log s) loses log s next to a huge m
        p = np.exp(logp)
        h = -np.where(p > 0, p * logp, 0.0 * log_s).sum(axis=1)
        ok = (targets >= 0) & (targets < x.shape[1])
        lp = np.where(ok, logp[np.arange(len(x)), np.where(ok, targets, 0)], np.nan)
        order = np.where(np.isnan(x), -np.inf, x)
        ids = np.argsort(-order, axis=1, kind="stable")[:, :top]
        return lp, h, ids, np.take_along_axis(logp, ids, axis=1)


def near(got, want, tol, what):
    got, want = got.double().cpu().numpy(), np.asarray(want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))  # infinities, NaN
    with np.errstate(invalid="ignore"):
        good = same | (np.abs(got - want) <= tol)
    assert good.all(), f"{what}: {got[~good][:4]} instead of {want[~good][:4]}"


def run(logits, targets=None, top=5, scale=1.0, workspace=None, calls=2, stream=None):
    rows, vocab = logits.shape
    if targets is None:
        targets = torch.arange(rows, dtype=torch.int32) * 7919 % vocab
    out = lambda *s, dt=torch.float32: torch.full(s, -77, dtype=dt, device="cuda")  # noqa: E731
    lp, h, tl = out(rows), out(rows), out(rows, top)
    ids = out(rows, top, dt=torch.int32)
    ws = workspace if workspace is not None else pkv.alloc_logprobs_workspace(rows, vocab, top)
    for _ in range(calls):
        pkv.token_logprobs(logits, targets.cuda(), lp, h, ids, tl, ws, scale=scale, stream=stream)
    torch.cuda.synchronize()
    return lp, h, ids, tl


def check(logits, targets=None, top=5, scale=1.0, **kw):
    rows, vocab = logits.shape
    if targets is None:
        targets = torch.arange(rows, dtype=torch.int32) * 7919 % vocab
    lp, h, ids, tl = run(logits, targets, top, scale, **kw)
    wl, wh, wi, wt = expected(logits.double().cpu().numpy(), targets.numpy(), top, scale)
    assert np.array_equal(ids.cpu().numpy(), wi), "top_ids"
    with np.errstate(invalid="ignore"):
        base = 2.0 ** -20 + vocab * 2.0 ** -34
        near(lp, wl, np.abs(wl) * 2.0 ** -22 + base, "logprobs")
        near(tl, wt, np.abs(wt) * 2.0 ** -22 + base, "top_logprobs")
        near(h, wh, (wh + 1) * (wh * 2.0 ** -22 + base), "entropy")


def normal(seed, rows, vocab, dtype, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(rows, vocab, generator=g, device="cuda") * spread).to(dtype)


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (7, 33), (3, 255), (2, 4095),
                                        (4, 4097), (1, 20011), (2, 50257), (1, 128256), (3, 151936), (9, 32000)])
def test_sizes(dtype, rows, vocab):
    for top in sorted({0, 1, min(5, vocab), min(32, vocab)}):
        check(normal(vocab + top, rows, vocab, dtype), top=top)


@pytest.mark.gpu
@BOTH
def test_many_rows(dtype):
    check(normal(1, 700, 3001, dtype), top=20)
    check(normal(2, 150, 40000, dtype), top=7)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("scale", [0.25, 1.0, 1.7, 20.0, 1e-6, 1e6])
def test_scales(dtype, scale):
    check(normal(3, 5, 6007, dtype), top=9, scale=scale)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_rows_at_any_element(dtype, offset):
    """Slices: rows that start at no 16-byte boundary, strides that are odd; NaN around them."""
    big = torch.full((6, 5021), float("nan"), dtype=dtype, device="cuda")
    big[:, offset:offset + 5000 - 3 * offset] = normal(4, 6, 5000 - 3 * offset, dtype)
    check(big[:, offset:offset + 5000 - 3 * offset], top=12)
    check(big[::2, offset:offset + 5], top=5)


@pytest.mark.gpu
@BOTH
def test_ties_and_orders(dtype):
    vocab = 30011
    rows = [torch.zeros(vocab), torch.arange(vocab).float() / 100, -torch.arange(vocab).float() / 100,
            (torch.arange(vocab) % 3).float(), (torch.arange(vocab) // 4096).float(),
            (torch.arange(vocab) % 4096).float(), -(torch.arange(vocab) % 4096 // 8).float()]
    near_top = torch.zeros(vocab)
    near_top[5000:5300] = 9.0  # more equals than alternatives, in neighbouring vectors
    strided = torch.zeros(vocab)
    strided[7::4096] = 5.0     # all in one thread's vectors
    strided[8::4096] = 5.5
    block = torch.randn(vocab, generator=torch.Generator().manual_seed(5))
    for j in range(8):         # whole groups of high, ascending values: more candidates than fit at once
        for t in range(32):
            at = torch.arange(8 * t + j, vocab, 4096)
            block[at] = 100 + torch.arange(len(at)).float() + t / 64 + j / 512
    zeros = torch.where(torch.arange(vocab) % 2 == 0, torch.tensor(0.0), torch.tensor(-0.0))
    x = torch.stack(rows + [near_top, strided, block, zeros]).to(dtype).cuda()
    for top in (1, 5, 32):
        check(x, top=top)


@pytest.mark.gpu
@BOTH
def test_masked_and_not_finite(dtype):
    vocab, inf, nan = 20000, float("inf"), float("nan")
    x = normal(6, 14, vocab, dtype)
    lowest = torch.finfo(dtype).min
    x[0, 3:] = -inf                        # three tokens allowed, fewer than the alternatives
    x[1, :19990] = -inf
    x[2] = -inf
    x[2, 777] = -5.0                       # one token: certain
    x[3] = -inf                            # none: no distribution
    x[4, 123] = nan
    x[5, 4000] = inf
    x[6, ::2] = lowest                     # masked by the lowest value
    x[7] = lowest                          # all of them: uniform
    x[8, 100:] = -inf
    x[8, :100] = lowest                    # uniform over the first hundred
    x[9] = nan
    x[10] = torch.finfo(dtype).max         # uniform again
    x[11] -= 30000.0 if dtype == torch.float32 else 1000.0
    x[12, 5] = 3000.0                      # far above the others
    x[13, :] = -inf
    x[13, 9], x[13, 10] = lowest, 0.0
    targets = torch.tensor([1, 5, 777, 0, 3, 3, 0, 3, 150, 3, 1, 2, 5, 9], dtype=torch.int32)
    check(x, targets, top=5)
    check(x, targets, top=32, scale=0.5 if dtype == torch.float32 else 1.0)


@pytest.mark.gpu
def test_targets_outside_the_vocabulary_have_no_logprob():
    targets = torch.tensor([-1, 0, 999, 1000, -2**31, 2**31 - 1], dtype=torch.int32)
    check(normal(7, 6, 1000, torch.bfloat16), targets)


@pytest.mark.gpu
def test_outputs_that_are_left_out():
    x = normal(8, 4, 9000, torch.float32)
    lp, h, ids, tl = run(x)
    ws = pkv.alloc_logprobs_workspace(4, 9000, 5)
    h2, ids2, tl2 = torch.empty_like(h), torch.empty_like(ids), torch.empty_like(tl)
    pkv.token_logprobs(x, None, None, h2, None, None, ws)
    pkv.token_logprobs(x, None, None, None, ids2, tl2, ws)
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(ids, ids2) and torch.equal(tl, tl2)


@pytest.mark.gpu
def test_the_same_bits_every_time():
    for rows, vocab in ((1, 128256), (3, 60000), (40, 128256)):
        x = normal(9, rows, vocab, torch.bfloat16)
        ws = pkv.alloc_logprobs_workspace(rows, vocab, 20)
        a = run(x, top=20, workspace=ws)
        for _ in range(5):
            assert all(torch.equal(s, t) for s, t in zip(a, run(x, top=20, workspace=ws)))


@pytest.mark.gpu
def test_a_workspace_serves_other_sizes():
    ws = pkv.alloc_logprobs_workspace(64, 50000, 32)
    for rows, vocab, top in ((64, 50000, 32), (1, 50000, 5), (7, 12345, 0), (64, 100, 3), (2, 50000, 20)):
        if pkv.token_logprobs_workspace_bytes(rows, vocab, top) <= ws.numel():
            check(normal(rows, rows, vocab, torch.bfloat16), top=top, workspace=ws)


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    big = torch.empty(3, 2**31 + 24, dtype=torch.bfloat16, device="cuda")[:, :7001]
    big.copy_(normal(10, 3, 7001, torch.bfloat16))
    check(big, top=5)


@pytest.mark.gpu
def test_another_stream_and_a_graph():
    x = normal(11, 3, 70000, torch.bfloat16)
    targets = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    want = run(x, targets.cpu(), top=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = pkv.alloc_logprobs_workspace(3, 70000, 8)
    got = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.token_logprobs(x, targets, *got, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals():
    lib, nan, inf = pkv.lib(), float("nan"), float("inf")
    # logits, type, stride, rows, vocab, scale, targets, top, logprobs, entropy, ids, top_logprobs, ws, bytes, stream
    good = [256, 0, 1000, 4, 1000, 1.0, 256, 5, 256, 256, 256, 256, 256, 1 << 30, None]
    for i, values in ((0, [None, 257]), (1, [2, -1]), (2, [-1]), (3, [-1]), (4, [0, -5, (1 << 30) + 1, 4]),
                      (5, [0.0, -1.0, nan, inf, 1e-7, 1e7]), (6, [None]), (7, [-1, 33]), (8, [None]), (10, [None]),
                      (11, [None]), (12, [None, 264])):
        for bad in values:
            args = list(good)
            args[i] = bad
            assert lib.token_logprobs(*args) == -22, (i, bad)
    args = list(good)
    args[3] = 0
    assert lib.token_logprobs(*args) == 0  # nothing to do
    for rows, vocab, top in ((0, 10, 1), (4, 0, 0), (4, 10, 11), (4, 100, 33), (4, 100, -1)):
        assert pkv.token_logprobs_workspace_bytes(rows, vocab, top) == 0
    x = torch.zeros(4, 100)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.token_logprobs(x, None, None, None, None, None, torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        pkv.token_logprobs(x[0], None, None, None, None, None, torch.zeros(1024, dtype=torch.uint8))


@pytest.mark.gpu
def test_binding_refusals():
    x = normal(12, 4, 100, torch.float32)
    ws = pkv.alloc_logprobs_workspace(4, 100, 5)
    f, i = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    ids, tl = torch.zeros(4, 5, dtype=torch.int32, device="cuda"), torch.zeros(4, 5, device="cuda")
    good = dict(logits=x, targets=i, logprobs=f, entropy=f.clone(), top_ids=ids, top_logprobs=tl, workspace=ws)
    for name, bad in (("logits", x.half()), ("logits", x.t().contiguous().t()), ("targets", i.long()),
                      ("targets", i[:3]), ("logprobs", f.double()), ("entropy", f[:2]), ("top_ids", ids.long()),
                      ("top_logprobs", tl[:, :4])):
        with pytest.raises(ValueError):
            pkv.token_logprobs(**{**good, name: bad})
    for name in ("targets", "logprobs", "top_logprobs"):
        with pytest.raises(pkv.PkvError, match="EINVAL"):
            pkv.token_logprobs(**{**good, name: None})
    with pytest.raises(pkv.PkvError, match="EINVAL"):
        pkv.token_logprobs(**{**good, "workspace": ws[:256].clone()})
