"""The example that runs the decoding-step operators and ConvTranspose together: replayed from a
graph it gives what single calls give, and its frames are the upsampler's input."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_graph_and_single_calls_agree():
    from examples.frame_decoder import CHANNELS, FrameDecoder, upsample
    a, b = (FrameDecoder(5, 40, width=256, layers=2, heads=8, kv_heads=2) for _ in range(2))
    for n in (3, 1, 20):
        x, y = a.generate(n, eager=True), b.generate(n)
        torch.cuda.synchronize()
        done = int(a.lengths[0])
        assert torch.equal(a.lengths, b.lengths) and torch.equal(x[:, :, :done], y[:, :, :done])
    assert done == 24 and x[:, :, :done].isfinite().all()
    # frames differ from step to step: the cache is read
    assert (x[:, :, 1:done] != x[:, :, :done - 1]).any(2).all()
    up = upsample(x[:, :, :done].contiguous())
    assert up.shape == (5, 64, 4 * done) and up.isfinite().all()
    assert x.shape[1] == CHANNELS
