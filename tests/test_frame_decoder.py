"""CPU tests of the frame decoder example's host side: which frames are single steps, and its room."""
import pytest
import torch

from examples.frame_decoder import FrameDecoder


class Counted(FrameDecoder):
    """A decoder whose steps only count themselves."""

    def __init__(self, frames):
        self.out, self.graph, self.steps = torch.zeros(2, 128, frames), None, 0

    def step(self):
        self.steps += 1


@pytest.mark.parametrize("eager", [False, True])
def test_one_frame_at_first(eager):
    """One frame before there is a graph is a single step."""
    m = Counted(4)
    assert m.generate(0, eager) is m.out and m.steps == 0
    assert m.generate(1, eager) is m.out and m.steps == 1
    m.generate(1, eager)
    assert m.steps == 2 and m.graph is None
