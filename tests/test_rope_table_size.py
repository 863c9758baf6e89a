"""A RoPE table's readers take its number of rows, and with it the place of its fp64
part, from its size: a table of other than the rows built is refused."""
import pytest
import torch

import paged_kv_decode_rope_gb300 as pkv


@pytest.mark.parametrize("size", [0, 9 * 1024, 10 * 1024 - 1, 10 * 1024 + 1, 11 * 1024, 20 * 1024])
def test_a_table_of_other_size_is_refused(size):
    with pytest.raises(ValueError, match="must hold num_positions = 10 rows"):
        pkv.paged_rope_table_build_freqs([1.0, 0.5], 10, torch.zeros(size, dtype=torch.uint8))


@pytest.mark.gpu
def test_the_fp64_part_is_where_the_append_reads_it():
    freqs, _ = pkv.rope_frequencies(10000.0)
    table = pkv.alloc_rope_table(100)
    pkv.paged_rope_table_build_freqs(freqs, 100, table)
    full = table[pkv.rope_table_rows(table) * 512:].view(torch.float64).view(100, 32, 2).cpu()
    angle = torch.arange(100, dtype=torch.float64)[:, None] * torch.tensor(freqs, dtype=torch.float64)
    assert float((full - torch.stack([angle.cos(), angle.sin()], -1)).abs().max()) < 1e-15
    with pytest.raises(ValueError, match="100 rows, got 101"):
        pkv.paged_rope_table_build_freqs(freqs, 100, pkv.alloc_rope_table(101))
