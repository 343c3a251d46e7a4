"""GPU tests of the frame decoder example: few frames at a time, and its room."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_single_frames_before_the_graph():
    """One frame at a time from the start, then more: the same frames as from single calls."""
    from examples.frame_decoder import FrameDecoder
    a, b = (FrameDecoder(3, 20, width=256, layers=1, heads=8, kv_heads=2) for _ in range(2))
    for n in (1, 1, 5, 1):
        x, y = a.generate(n, eager=True), b.generate(n)
        torch.cuda.synchronize()
        done = int(a.lengths[0])
        assert torch.equal(a.lengths, b.lengths) and torch.equal(x[:, :, :done], y[:, :, :done])
    assert done == 8 and b.graph is not None
