"""What the binding of the operators over a vocabulary makes of a table's shape, with a
recorder in the library's place: needs no GPU."""

import pytest
import torch

q = pytest.importorskip("quantized_weight_backward_amd")
from quantized_weight_backward_amd import vocab  # noqa: E402


@pytest.fixture
def table(monkeypatch):
    monkeypatch.setattr(vocab, "_device_tensor", lambda t, name, contiguous=True: t)
    return vocab._table


def bytes_of(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def test_rows_of_a_contiguous_table_wider_than_its_blocks(table):
    """A 2-D uint8 table has the rows that its shape says: padding is no row."""
    for width in (34, 36, 68, 102, 340):
        assert table(q.Q8_0, bytes_of(9, width), 32) == (9, width)
    assert table(q.Q4_K, bytes_of(5, 2 * 144), 256) == (5, 288)
    assert table(q.MXFP4, bytes_of(5, 18), 32) == (5, 18)
    assert table(q.F32, bytes_of(5, 64), 8) == (5, 64)
    # one row: what is behind it is not a distance between rows
    assert table(q.Q8_0, bytes_of(1, 35), 32) == (1, 34)
    assert table(q.Q8_0, bytes_of(0, 68), 32)[0] == 0


def test_tables_of_bytes_alone(table):
    """Other contiguous tensors hold N row_bytes bytes in whatever shape."""
    assert table(q.Q8_0, bytes_of(9 * 34), 32) == (9, 34)
    assert table(q.Q8_0, bytes_of(3, 3, 34), 32) == (9, 34)
    assert table(q.Q8_0, bytes_of(18, 17), 32) == (9, 34)  # no row of it holds a row of the table
    assert table(q.BF16, torch.zeros(6, 8, dtype=torch.bfloat16), 8) == (6, 16)
    for W in (bytes_of(35), bytes_of(18, 33)):
        with pytest.raises(ValueError):
            table(q.Q8_0, W, 64)


def test_views(table):
    wide = bytes_of(9, 100)
    assert table(q.Q8_0, wide[:, :34], 32) == (9, 100)
    assert table(q.Q8_0, wide[:, 2:80], 32) == (9, 100)
    assert table(q.Q8_0, wide[::2, :34], 32) == (5, 200)
    for W in (wide[:, :33], wide.T, wide.view(torch.int16)[:, :20], wide[:, ::2], wide[:1, ::2]):
        with pytest.raises(ValueError):
            table(q.Q8_0, W, 32)
