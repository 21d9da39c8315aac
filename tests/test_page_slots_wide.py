"""page_slots with 64-bit tables: entries whose slot passes 64 bits as well."""
import pytest
import torch

import varlen_top_select_amd as vts


@pytest.mark.parametrize("page_size,entry", [(16, 2 ** 60), (16, 2 ** 60 + 5), (4, 2 ** 62), (64, 3 * 2 ** 58 + 1),
                                             (2 ** 31, 2 ** 33), (3, 2 ** 63 - 1), (16, 2 ** 31)])
def test_entries_past_64_bits(page_size, entry):
    """No slot, where their product with page_size wrapped to another page's."""
    table = torch.tensor([[entry, 7], [3, entry]])
    pos = torch.tensor([[0, page_size, 2], [1, page_size, page_size + 2]])
    got = vts.page_slots(table, page_size, pos)
    known = page_size < 2 ** 20
    assert got.tolist() == [[-1, 7 * page_size if known else -1, -1], [3 * page_size + 1 if known else -1, -1, -1]]


def test_large_pages():
    """A page of 2^31 positions has slots of its first 2^31 - 1 alone."""
    pos = torch.tensor([[0, 2 ** 31 - 1, 2 ** 31, 2 ** 40]])
    assert vts.page_slots(torch.tensor([[0]]), 2 ** 31, pos).tolist() == [[0, 2 ** 31 - 1, -1, -1]]
    assert vts.page_slots(torch.tensor([[0, 1]]), 2 ** 40, pos).tolist() == [[0, 2 ** 31 - 1, -1, -1]]
