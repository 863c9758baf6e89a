"""Windows that begin inside the shared pages, in the kernel for shared pages (every
test sees that it ran), and values that are not finite where only some members of a
group see them. Formula and tolerances: test_gpu_decode_shared.py."""
import math

import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv
from tests.test_gpu_decode_shared import PAGE, Batch

LONG = 2048 * PAGE + 5  # more pages than the kernel for little work takes


@pytest.fixture(autouse=True)
def tables_as_narrow_as_they_can_be():
    Batch.least_cols = 0


def run(b, dtype, **kw):
    """The call, and that it wrote the workspace, which the kernel for little work does not."""
    ws = pkv.alloc_shared_workspace(len(b.lens), b.hq, b.hkv)
    ws.fill_(255)
    got = b.run(dtype, ws, **kw)
    assert bool((ws[:16 * (len(b.lens) + 1)] != 255).any())
    again = b.run(dtype, ws, **kw)
    assert torch.equal(got.view(torch.int16 if dtype == torch.bfloat16 else torch.int32),
                       again.view(torch.int16 if dtype == torch.bfloat16 else torch.int32))
    return got


def slopes_of(b):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / b.hq) for i in range(b.hq)], device="cuda")


def check(b, dtype=torch.float32, softcap=0.0, alibi=False, bits=0):
    """Within the tolerance where the definition is finite, not finite where it is not."""
    slopes = slopes_of(b) if alibi else None
    got = run(b, dtype, softcap=softcap, alibi_slopes=slopes)
    want, tol = b.want(softcap, slopes, dtype)
    assert pkv.pkv_get_error(b.pool, reset=True) == bits
    fine = want.isfinite()
    assert torch.equal(got.isfinite(), fine)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    limit = tol + half * (want.abs() + tol) + 1e-38
    assert bool(((got.double() - want).abs() <= limit)[fine].all())
    return fine


def nan_before(b, shared):
    """NaN in the slots of the shared pages before the first key that anyone sees."""
    first = min(lo for n, lo in zip(b.lens, b.lo) if n > 0)
    if first // PAGE < shared // PAGE and first % PAGE:
        b.storage[b.tables[0, first // PAGE].long(), :, :, :first % PAGE] = math.nan


SCORES = [(0.0, False), (20.0, False), (0.0, True), (5.0, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softcap,alibi", SCORES)
@pytest.mark.parametrize("hq,hkv,past", [
    (8, 2, [0, 1, 15, 16, 17, 63, 64, 65]), (14, 2, [1, 1, 1]), (3, 3, [16, 32, 48]), (8, 1, [63, 200]), (4, 4, [79, 80, 81, 700]),
    (16, 2, [129 + 16 * i for i in range(18)])])
def test_few_members_of_long_windows(hq, hkv, past, softcap, alibi, dtype):
    b = Batch(hq, hkv, [(LONG - 1, [LONG + i for i in past])], hq, LONG)
    nan_before(b, LONG)
    assert bool(check(b, dtype, softcap, alibi).all())
    b.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softcap,alibi", SCORES)
@pytest.mark.parametrize("window,least,most", [(300, 600, 640), (300, 601, 900), (257, 640, 2000), (320, 100, 700)])
def test_many_members_of_short_windows(window, least, most, softcap, alibi, dtype):
    g = torch.Generator().manual_seed(window + least)
    lens = torch.randint(least, most + 1, (260,), generator=g).tolist()
    b = Batch(16, 8, [(600, lens), (None, [window + 40])], 3, window)
    assert bool(check(b, dtype, softcap, alibi).all())
    b.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (5.0, True)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_some_members_see(value, softcap, alibi, dtype):
    """An old key's value that is not finite reaches the members whose window holds it, and no others."""
    b = Batch(8, 2, [(LONG - 1, [LONG + i for i in (3, 20, 40, 100, 900)])], 7, LONG)
    keep = b.storage.clone()
    for keys in ((10,), (3, 19, 20), (39, 99, 150), (899, 500), (LONG - 40,)):
        for i, key in enumerate(keys):
            b.storage[b.tables[min(range(5), key=lambda m: b.lo[m]), key // PAGE].long(), i % 2, 1, key % PAGE, 7 * i:7 * i + 3] = value
        fine = check(b, dtype, softcap, alibi)
        sees = torch.tensor([any(lo <= key for key in keys) for lo in b.lo], device="cuda")
        assert torch.equal(~fine.flatten(1).all(-1), sees)
        b.storage.copy_(keep)
    b.storage[b.tables[0, 30 // PAGE].long(), :, 0, 30 % PAGE, 5] = math.nan  # of a key: every weight of those who see it
    check(b, dtype, softcap, alibi)
    b.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_that_some_of_many_members_see(dtype):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(600, 900, (150,), generator=g).tolist()
    b = Batch(32, 8, [(600, lens), (48, [300, 301, 310] * 20)], 4, 290)
    where = (b.storage.new_ones(b.storage.shape[:4]).float().uniform_(generator=torch.Generator(device="cuda").manual_seed(1)) < 2e-3)
    b.storage[..., 1, :, 9] = torch.where(where[:, :, 1], math.inf, b.storage[..., 1, :, 9].float()).to(torch.bfloat16)
    b.storage[..., 1, :, 40] = torch.where(where[:, :, 0], math.nan, b.storage[..., 1, :, 40].float()).to(torch.bfloat16)
    fine = check(b, dtype)
    assert not bool(fine.all()) and bool(fine[:, :, 10:40].all()) and bool(fine[:, 0].any())
    b.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, LONG])
def test_members_of_bad_lengths_beside_values_that_are_not_finite(window):
    b = Batch(8, 2, [(LONG - 1, [LONG + 30, LONG + 90, LONG + 5])], 2, window)
    b.storage[b.tables[2, 100].long(), :, 1, 3, 4] = math.nan
    for bad in (0, -5, b.cols * PAGE + 1, -2**31, 2**31 - 1):
        b.lens[1] = bad
        b.seq_lens = torch.tensor(b.lens, dtype=torch.int32, device="cuda")
        fine = check(b, bits=pkv.ERR_SEQ_LEN)
        assert fine[1].all() and not bool(fine[0, :, 4].any()) and bool(fine[0, :, 5].all())
    b.pool.close()
