"""CPU tests of tree_mask on parents that are no draft of the tree."""
import pytest
import torch

import convt_forward_amd as C


@pytest.mark.parametrize("stray", [3, 4, 63, 64, 2 ** 40, 2 ** 63 - 1, -2, -2 ** 63])
def test_a_parent_that_is_no_draft_is_the_cached_tokens(stray):
    parents = torch.tensor([[-1, 0, stray], [2, stray, 1]])
    want = C.tree_mask(torch.tensor([[-1, 0, -1], [2, -1, 1]]))
    assert torch.equal(C.tree_mask(parents), want)
    assert torch.equal(C.tree_mask(parents.transpose(0, 1).contiguous().transpose(0, 1)), want)


def test_loops_and_no_drafts():
    # drafts that follow each other see each other
    assert C.tree_mask(torch.tensor([1, 0, 2])).flatten().tolist() == [3, 3, 4]
    assert C.tree_mask(torch.zeros(2, 0, dtype=torch.int64)).shape == (2, 0, 0)
