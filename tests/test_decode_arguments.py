"""Arguments of the decode-step operators at their edges, without a GPU."""
import pytest
import torch

import varlen_top_select_amd as vts


@pytest.mark.parametrize("bad", [4, 5, 64, 2 ** 31 - 1, -2, -2 ** 31])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_tree_mask_of_parents_that_are_no_node(bad, dtype):
    """A node whose parent does not exist (verify_draft never accepts it) sees
    itself, and no entry past the row is looked up."""
    parents = torch.tensor([[-1, bad, 1, 0], [bad, 0, 1, bad]], dtype=dtype)
    assert vts.tree_mask_from_parents(parents).tolist() == [[1, 2, 6, 9], [1, 3, 7, 8]]


def test_tree_mask_of_no_tokens():
    assert vts.tree_mask_from_parents(torch.empty(3, 0, dtype=torch.int32)).shape == (3, 0)
    assert vts.tree_mask_from_parents(torch.empty(0, 5, dtype=torch.int32)).shape == (0, 5)
