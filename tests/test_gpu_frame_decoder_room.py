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


def test_no_room_after_replays():
    """Frames replayed from the graph count too: the one past the room is refused, and nothing is enqueued for it."""
    from examples.frame_decoder import FrameDecoder
    m = FrameDecoder(2, 6, width=256, layers=1, heads=8, kv_heads=2)
    m.generate(4)
    with pytest.raises(ValueError, match="room"):
        m.generate(3)
    x = m.generate(2)
    torch.cuda.synchronize()
    assert m.lengths.tolist() == [6, 6] and m.done == 6 and x.isfinite().all()
    for eager in (False, True):
        with pytest.raises(ValueError, match="room"):
            m.generate(1, eager)
    torch.cuda.synchronize()
    assert m.lengths.tolist() == [6, 6]
