"""GPU tests of the operators of several new tokens at the ends of their number ranges: values near the
largest of their type."""
import pytest
import torch

import convt_forward_amd as C
from tests.decode_util import within
from tests.extend_util import DEV, Streams, attend64, row_bound, tree_seen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("route", ["direct", "auto"])
@pytest.mark.parametrize("form", ["few rows", "128 rows", "256 rows"])
def test_values_near_the_largest(form, route):
    """A token whose score passes those before it by 2^7.2, less than what moves the base of the
    exponents, holds values near bfloat16's largest; all others hold zeros, and the result is finite."""
    batch, kv, drafts, share, room = {"few rows": (2, 1, 2, 4, 300), "128 rows": (2, 1, 25, 4, 300), "256 rows": (4, 8, 64, 4, 4700)}[form]
    s = Streams(batch, room, kv, 64, 16, "bf16", False, seed=90)
    for name in "kv":
        s.host[name].zero_()
    lengths = [room - drafts - 10 * b for b in range(batch)]
    at = 144  # in a later tile than the first one, of the same wave in the form for few rows too: its tiles of 32 tokens go round 4 waves
    for b in range(batch):
        page, off = int(s.table[b, at // 16]), at % 16
        s.host["k"][page, :, off, 0] = 5.0
        s.host["v"][page, :, off] = (torch.linspace(-1, 1, 64) * 3e38).bfloat16()
    for name in "kv":
        getattr(s.cache, name).copy_(s.host[name].to(DEV))
    q = torch.zeros(batch, drafts, kv * share, 64, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    tree = C.tree_mask(torch.arange(-1, drafts - 1))
    got, lse = C.tree_attention(q.to(DEV), s.cache, s.table.to(DEV), torch.tensor(lengths, dtype=torch.int32, device=DEV), tree.to(DEV), scale=1.0,
                                lse=True, route=route)
    torch.cuda.synchronize()
    k, v = s.tokens64("k"), s.tokens64("v")
    for b in range(batch):
        seen = tree_seen(lengths[b], drafts, s.room, tree.tolist())[[0, drafts - 1]]
        want, want_lse, mag, top = attend64(q[b][[0, drafts - 1]], k[b], v[b], seen, 1.0)
        assert want.isfinite().all() and want.abs().max() > 1e36
        step = 0.0 if route == "direct" else 2.0 ** -8
        within(got[b][[0, drafts - 1]], want, row_bound(want, mag, top, 64, s.room, "bf16", step, False), f"stream {b}")
