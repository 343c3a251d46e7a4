"""GPU tests of window_attention's forms and parts on ragged batches, each row that is looked at held to
its own bound in 64 bits (sum p |V| and the weights' step): a part that is lost, or joined with a wrong
factor, shows in rows over thousands of tokens too."""
import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import TYPES, U, within
from tests.extend_util import DEV, Streams, attend64, p_step, rand, row_bound, window_seen

pytestmark = pytest.mark.gpu


def check(s, lengths, news, heads, window, sinks, route="auto"):
    t = TYPES[s.dt]
    q = rand(sum(news) + 3, heads, s.dim, seed=1, scale=2).to(t)
    starts = torch.tensor([0] + news).cumsum(0).to(torch.int32)
    out = torch.full(q.shape, 3.0, dtype=t, device=DEV)
    got, lse = C.window_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), starts=starts.to(DEV),
                                  window=window, sinks=sinks, out=out, lse=True, route=route)
    torch.cuda.synchronize()
    assert (out[sum(news):] == 3).all()
    k, v = s.tokens64("k"), s.tokens64("v")
    step = p_step(s.dt, s.cache.quantised, "direct" if route == "direct" else "mfma")
    for b, n in enumerate(news):
        if n == 0:
            continue
        pick = sorted({0, 1 % n, n // 3, n // 2, n - 1})
        seen = window_seen(lengths[b], n, s.room, window, sinks)[pick]
        r = [int(starts[b]) + i for i in pick]
        want, want_lse, mag, top = attend64(q[r], k[b], v[b], seen, s.dim ** -0.5)
        most = int(seen.sum(1).max())
        within(got[r], want, row_bound(want, mag, top, s.dim, most, s.dt, step, s.cache.quantised), f"stream {b}, {n} new of {lengths[b]}")
        within(lse[r], want_lse, 2 * (s.dim + 12) * U * top + (most + 64) * U + 2.0 ** -17 + want_lse.abs().nan_to_num(0, 0, 0) * 4 * U, f"lse {b}")


@pytest.mark.parametrize("window,sinks", [(None, 0), (3000, 70), (100, 2)])
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("bf16", True), ("f16", False), ("f16", True)])
@pytest.mark.parametrize("new,share", [(1, 4), (7, 4), (20, 4), (60, 4), (150, 2), (300, 8)])
def test_one_long_stream_among_short_ones(new, share, dt, quantised, window, sinks):
    s = Streams(4, 5000, 1, 64, 16, dt, quantised, seed=new)
    check(s, [4990, 0, max(new // 2, 40), 900], [new, 0, new // 2, new], share, window, sinks)


@pytest.mark.parametrize("route", ["direct", "auto"])
@pytest.mark.parametrize("dt,quantised", [("bf16", False), ("bf16", True)])
@pytest.mark.parametrize("at", [0, 31, 63])
def test_a_chunk_among_single_tokens(at, dt, quantised, route):
    """63 streams with one new token and one with a chunk of a prompt, in front of, among and behind them."""
    s = Streams(64, 700, 1, 64, 16, dt, quantised, seed=99)
    news = [1] * 64
    news[at] = 256
    lengths = [700 - 11 * b for b in range(64)]
    lengths[at] = 600
    for window, sinks in ((None, 0), (200, 4)):
        check(s, lengths, news, 4, window, sinks, route)
