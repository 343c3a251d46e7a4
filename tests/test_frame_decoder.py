"""CPU tests of the frame decoder example's host side: which frames are single steps, and its room."""
import pytest
import torch

from examples.frame_decoder import FrameDecoder


class Counted(FrameDecoder):
    """A decoder whose steps only count themselves."""

    def __init__(self, frames):
        self.out, self.graph, self.done, self.steps = torch.zeros(2, 128, frames), None, 0, 0

    def enqueue(self):
        self.steps += 1


@pytest.mark.parametrize("eager", [False, True])
def test_one_frame_at_first(eager):
    """One frame before there is a graph is a single step."""
    m = Counted(4)
    assert m.generate(0, eager) is m.out and m.steps == 0
    assert m.generate(1, eager) is m.out and m.steps == 1
    m.generate(1, eager)
    assert m.steps == 2 and m.graph is None


@pytest.mark.parametrize("eager", [False, True])
def test_no_room_is_refused_on_the_host(eager):
    """More frames than have room are refused before any of them is enqueued, and those that have it still run."""
    m = Counted(3)
    for n in (4, 100):
        with pytest.raises(ValueError, match="room"):
            m.generate(n, eager)
    assert m.steps == 0
    m.generate(1, eager)
    m.step()
    with pytest.raises(ValueError, match="room"):
        m.generate(2, eager)
    m.generate(1, eager)
    assert m.steps == m.done == 3
    for bad in (lambda: m.generate(1, eager), m.step):
        with pytest.raises(ValueError, match="room"):
            bad()
    assert m.generate(0, eager) is m.out and m.steps == 3
