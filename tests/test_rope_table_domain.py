"""The cos and sin of a RoPE table are worked out for angles below 2^52: frequencies
that lead past it are refused (the reduction would give any number)."""
import ctypes

import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv


def call(freqs, rows, at=256):
    arr = (ctypes.c_double * len(freqs))(*freqs)
    return pkv.lib().paged_rope_table_build_freqs(arr, len(freqs), 1.0, rows, at, None)


@pytest.mark.skipif(torch.cuda.is_available(), reason="an address that is no memory; no launch can happen here")
def test_angles_past_the_reduction_are_refused():
    most = 2.0 ** 52
    for f in (most, -most, 1e300, -1e300):
        assert call([1.0, f], 2) == -22
        assert call([1.0, f / 1023], 1024) == -22
        assert call([f], 1) == -5  # position 0 alone has angle 0: not refused, the launch fails without a GPU
    for f in (most * (1 - 2.0 ** -53), -most * (1 - 2.0 ** -53)):
        assert call([1.0, f], 2) == -5
        assert call([1.0, f / 1024], 1025) == -5


@pytest.mark.gpu
def test_the_largest_angles():
    freqs = [2.0 ** 40 + 0.5, -(2.0 ** 41), 3.0e12, 1.0]
    table = pkv.alloc_rope_table(1000)
    pkv.paged_rope_table_build_freqs(freqs, 1000, table)
    full = table[1000 * 512:].view(torch.float64).view(1000, 32, 2).cpu()[:, :4]
    angle = torch.arange(1000, dtype=torch.float64)[:, None] * torch.tensor(freqs, dtype=torch.float64)
    # the C library reduces any argument; an ulp of it and half a one of the table's
    assert float((full - torch.stack([angle.cos(), angle.sin()], -1)).abs().max()) <= 2.0 ** -51
