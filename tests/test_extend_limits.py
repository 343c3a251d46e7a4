"""CPU tests of the limits of the attention of several new tokens: queries only, nothing is launched."""
import pytest

from tests.test_extend_abi import tree_query, window_query


@pytest.mark.parametrize("batch", [2 ** 24, 2 ** 30 + 1, 2 ** 31 - 65, 2 ** 31 - 1])
def test_too_many_streams(batch):
    # the kernels' searches add to and halve indexes of streams in 32 bits, also of streams without rows
    assert window_query(batch=batch, tokens=4, ragged=1)[0] == 2
    assert window_query(batch=batch, tokens=0, ragged=1)[0] == 2
    assert tree_query(batch=batch, drafts=1)[0] == 2


def test_most_streams():
    assert window_query(batch=2 ** 24 - 1, tokens=4, ragged=1)[0] == 0
    assert window_query(batch=2 ** 22 - 1, tokens=2 ** 22 - 1)[0] == 0
