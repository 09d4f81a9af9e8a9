"""The paged binding's checks of shapes and numbers that sit at an edge, on the CPU."""
import pytest
import torch

from split_kv_decode_decoding_gb300 import paged


def test_a_table_of_one_page_has_rows_of_any_stride():
    """[B, 1] as a transposed row or a column of a wider tensor: its rows are one entry each, and contiguous."""
    paged._init()
    lens = torch.ones(3, dtype=torch.int32)
    for table, stride in ((torch.arange(3, dtype=torch.int32).view(1, 3).t(), 1), (torch.zeros(3, 5, dtype=torch.int32)[:, 2:3], 5),
                          (torch.zeros(3, 1, 4, dtype=torch.int32)[:, :, 1], 4)):
        assert table.shape == (3, 1)
        assert paged._check_sequences(lens, table, -1) == (3, 1, stride)
    with pytest.raises(ValueError):
        paged._check_sequences(lens, torch.zeros(2, 3, dtype=torch.int32).t(), -1)
