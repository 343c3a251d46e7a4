"""GPU tests of calls of the attention and append operators that have to be refused: numbers that the
C structs cannot hold."""
import pytest
import torch

import convt_forward_amd as C
from tests.extend_util import DEV, Streams, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_length", [2 ** 64 + 100, 2 ** 64, 2 ** 63, 2 ** 62, 2 ** 31, -2 ** 63 - 1, -2 ** 64, -1])
def test_max_length_beyond_64_bits(max_length):
    s = Streams(2, 200, 1, 64, 16, "bf16", False, seed=95)
    q, table, lengths = rand(2, 4, 64).bfloat16().to(DEV), s.table.to(DEV), torch.tensor([150, 20], dtype=torch.int32, device=DEV)
    tree = C.tree_mask(torch.tensor([-1])).to(DEV)
    with pytest.raises(C.ConvtError):
        C.window_attention(q, s.cache, table, lengths, max_length=max_length)
    with pytest.raises(C.ConvtError):
        C.tree_attention(q.view(2, 1, 4, 64), s.cache, table, lengths, tree, max_length=max_length)


@pytest.mark.parametrize("max_length", [2 ** 64 + 100, 2 ** 64, 2 ** 63, -2 ** 64])
def test_max_length_of_one_token_beyond_64_bits(max_length):
    s = Streams(2, 200, 1, 64, 16, "bf16", False, seed=95)
    q, lengths = rand(2, 4, 64).bfloat16().to(DEV), torch.tensor([150, 20], dtype=torch.int32, device=DEV)
    with pytest.raises(C.ConvtError):
        C.decode_attention(q, s.cache, s.table.to(DEV), lengths, max_length=max_length)


def test_windows_and_sinks_beyond_64_bits_are_all_there_is():
    s = Streams(2, 200, 1, 64, 16, "bf16", False, seed=96)
    q, table, lengths = rand(2, 4, 64).bfloat16().to(DEV), s.table.to(DEV), torch.tensor([150, 20], dtype=torch.int32, device=DEV)
    want = C.window_attention(q, s.cache, table, lengths)
    assert torch.equal(C.window_attention(q, s.cache, table, lengths, window=2 ** 64 + 3), want)
    assert torch.equal(C.window_attention(q, s.cache, table, lengths, window=3, sinks=2 ** 64 + 1), want)
    for kw in (dict(window=-2 ** 64 + 5), dict(window=-2 ** 63)):
        with pytest.raises(ValueError):
            C.window_attention(q, s.cache, table, lengths, **kw)
    with pytest.raises(C.ConvtError):
        C.window_attention(q, s.cache, table, lengths, sinks=-2 ** 64 + 5)


def test_more_than_32_bits_of_heads_streams_or_drafts():
    """By strides of 0, so without their memory: none of these may be cut to their lowest 32 bits."""
    s = Streams(1, 32, 1, 64, 16, "bf16", False, seed=97)
    table, lengths, many = s.table.to(DEV), torch.tensor([20], dtype=torch.int32, device=DEV), 2 ** 32 + 4
    one = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    slots, inv = torch.zeros(1, dtype=torch.int64, device=DEV), torch.ones(32, device=DEV)
    tree = torch.ones(1, 1, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        C.cache_append(s.cache, one, one, slots, slots, inv, q=one.expand(1, many, 64))
    with pytest.raises(ValueError):
        C.window_attention(one.expand(1, many, 64), s.cache, table, lengths)
    with pytest.raises(ValueError):
        C.window_attention(one, s.cache, table.expand(2 ** 32 + 1, -1), lengths, starts=torch.tensor([0, 1], dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        C.tree_attention(one.view(1, 1, 1, 64).expand(1, 1, many, 64), s.cache, table, lengths, tree)
    with pytest.raises(ValueError):
        C.tree_attention(one.view(1, 1, 1, 64).expand(2 ** 32 + 1, 1, 1, 64), s.cache, table.expand(2 ** 32 + 1, -1), lengths, tree)
