"""CPU tests of the decoding-step operators at the edges of what they accept: the split of the
longest lengths, and the Python binding's checks, none of which needs a device."""
import ctypes

import pytest
import torch

import convt_forward_amd as C
from convt_forward_amd import decode as D


def attend_query(max_length, batch=1, heads=1, kv_heads=1, page=2 ** 20, dim=16, table_width=2048, table_stride=2048):
    strides = (ctypes.c_int64 * 3)(kv_heads * page * dim, page * dim, dim)
    cache = D.CacheDesc(1, strides, strides, kv_heads, page, dim, 1, 0, 0)
    two = (ctypes.c_int64 * 2)(heads * dim, dim)
    p = D.AttendProblem(cache, max_length, two, two, table_width, table_stride, batch, heads, 0, 1.0)
    info = D.AttendInfo()
    return D.lib().convt_attend_query(ctypes.byref(p), ctypes.byref(info)), info


@pytest.mark.parametrize("batch", [1, 40, 3000])
@pytest.mark.parametrize("length", [2 ** 30 + 1, 2 ** 31 - 2 ** 16, 2 ** 31 - 2 ** 16 + 1, 2 ** 31 - 4097])
def test_parts_of_the_longest_lengths(length, batch):
    """Up to the longest length accepted the parts cover it, and the first token of every part is
    an index of 31 bits; one more is refused."""
    st, i = attend_query(length, batch)
    assert st == 0 and 1 <= i.chunks <= 32768
    assert i.chunks == (length - 1) // i.chunk_tokens + 1
    assert (i.chunks - 1) * i.chunk_tokens < 2 ** 31
    assert attend_query(2 ** 31 - 4096, batch)[0] == 1


@pytest.mark.parametrize("shape", [(2, 0, 8), (0, 2, 8), (3, 0, 4, 8), (2, 3, 0, 8), (0, 0, 8), (0, 8)])
def test_no_rows_in_any_axis(shape):
    assert D._rows(torch.zeros(shape), "t")[0] == 0
    assert D._rows(torch.zeros(shape)[..., 2:5], "t")[0] == 0


def test_workspace_is_the_callers_whole_memory():
    """A workspace whose elements lie in less memory than they count, or on another device, is refused."""
    here = torch.device("cpu")
    D._check_workspace(torch.empty(64, dtype=torch.uint8), 64, here)
    D._check_workspace(torch.empty(200, dtype=torch.uint8)[100:], 64, here)
    D._check_workspace(torch.empty(4, 4), 64, here)
    for bad, why in [(torch.empty(1, dtype=torch.uint8).expand(64), "contiguous"), (torch.empty(128, dtype=torch.uint8)[::2], "contiguous"),
                     (torch.empty(63, dtype=torch.uint8), "too small"), (torch.empty(64, dtype=torch.uint8, device="meta"), "is on meta")]:
        with pytest.raises(ValueError, match=why):
            D._check_workspace(bad, 64, here)


def test_rows_that_are_only_read_may_repeat():
    """A stride of 0 is taken for x and page tables, and refused for what is written."""
    route = ctypes.c_int32()
    for xs, ys, want in ((0, 5, 0), (64, 5, 0), (0, 0, 1), (1, 5, 1), (-1, 5, 1)):
        p = D.Q4Problem(3, 5, 64, 32, xs, ys, 1, 0, 0, 0)
        assert D.lib().convt_q4_query(ctypes.byref(p), ctypes.byref(route)) == want, (xs, ys)
    assert [attend_query(100, batch=2, table_stride=s)[0] for s in (0, 2048, 1, 2047, -1)] == [0, 0, 1, 1, 1]


def fake_cache(monkeypatch, *shape, quantised=False):
    """A KVCache whose tensors lie on the CPU; only calls that launch nothing are made of it."""
    monkeypatch.setattr(D, "_check", lambda *a, **k: None)
    scales = [torch.zeros(shape[:3]) for _ in range(2)] if quantised else [None, None]
    kind = D._E4M3 if quantised else torch.bfloat16
    return C.KVCache(*(torch.zeros(shape, dtype=torch.uint8).to(kind) for _ in range(2)), *scales)


@pytest.mark.parametrize("quantised", [False, True])
def test_cache_follows_its_tensors(monkeypatch, quantised):
    """A tensor put in the place of another is checked like the first, and calls see its strides."""
    cache = fake_cache(monkeypatch, 4, 2, 16, 64, quantised=quantised)
    assert list(cache._desc(torch.bfloat16, "k").k_stride) == [2048, 1024, 64]
    q, table = torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 4, dtype=torch.int32)
    assert list(C.attend_plan(cache, q, table)[0].cache.k_stride) == [2048, 1024, 64]
    other = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).to(cache.k.dtype).transpose(1, 2)
    cache.k = other
    assert cache.k is other and list(cache._desc(torch.bfloat16, "k").k_stride) == [2048, 64, 128]
    assert list(cache._desc(torch.bfloat16, "k").v_stride) == [2048, 1024, 64]
    assert list(C.attend_plan(cache, q, table)[0].cache.k_stride) == [2048, 64, 128]
    with pytest.raises(ValueError):
        cache.v = other.permute(0, 1, 3, 2)  # its last axis is not contiguous
    with pytest.raises(ValueError):
        cache.k_scale = None if quantised else torch.zeros(4, 2, 16)
    for name in ("quantised", "n_pages", "kv_heads", "page_size", "head_dim", "device", "other"):
        with pytest.raises(AttributeError, match="KVCache"):
            setattr(cache, name, 1)
    assert cache.k is other and cache.quantised == quantised


def test_plan_goes_by_the_value_of_its_arguments(monkeypatch):
    """A scale or length given as a tensor counts with the value it has at the call."""
    cache = fake_cache(monkeypatch, 4, 2, 16, 64)
    q, table = torch.zeros(3, 4, 64).bfloat16(), torch.zeros(3, 4, dtype=torch.int32)
    scale, most = torch.tensor(0.5), torch.tensor(40)
    assert (lambda p: (p.scale, p.max_length))(C.attend_plan(cache, q, table, scale, most)[0]) == (0.5, 40)
    scale.fill_(0.25), most.fill_(50)
    assert (lambda p: (p.scale, p.max_length))(C.attend_plan(cache, q, table, scale, most)[0]) == (0.25, 50)
    assert C.attend_plan(cache, q, table, 0.25, 50)[0].max_length == 50
    with pytest.raises(TypeError):
        C.attend_plan(cache, q, table, 0.25, 50.0)


class Elsewhere:
    """A stand-in for a tensor of a second GPU: everything but its device is the CPU tensor's."""

    def __init__(self, t):
        self.t, self.device, self.is_cuda = t, torch.device("cuda", 1), True

    def __getattr__(self, name):
        return getattr(self.t, name)


class FakeDevices:
    """Keeps the current device, and the one that was current at each call of the library."""

    def __init__(self):
        self.now, self.calls = 0, []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, self.now)) or 0


@pytest.fixture
def two_devices(monkeypatch):
    fake = FakeDevices()

    class Context:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, fake.now = fake.now, self.index

        def __exit__(self, *a):
            fake.now = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: fake.now)
    monkeypatch.setattr(torch.cuda, "device", Context)
    monkeypatch.setattr(C, "_one_device", False)
    for module in (C, D):
        monkeypatch.setattr(module, "_launch_stream", lambda stream, device: (0, None))
    monkeypatch.setattr(D, "_empty", lambda shape, dtype, device: Elsewhere(torch.empty(tuple(shape), dtype=dtype)))
    return fake


def test_calls_go_to_their_tensors_device(two_devices, monkeypatch):
    """With device 0 current, calls on tensors of device 1 are launched there, and leave device 0 current."""
    C.lib(), D.lib()
    monkeypatch.setattr(D, "_ready", two_devices)
    t = lambda *shape, dtype=torch.bfloat16: Elsewhere(torch.zeros(*shape, dtype=dtype))  # noqa: E731
    cache = C.KVCache(t(4, 2, 16, 64), t(4, 2, 16, 64))
    C.rms_norm(t(3, 64), t(64))
    C.cache_write(cache, t(3, 2, 64), t(3, 2, 64), t(3, dtype=torch.int64))
    C.cache_read(cache, t(3, dtype=torch.int64))
    C.decode_attention(t(1, 4, 64), cache, t(1, 4, dtype=torch.int32), t(1, dtype=torch.int32))
    C.q4_matvec(t(3, 64), t(5, 32, dtype=torch.uint8), t(5, 2))
    assert [c for c in two_devices.calls if c[0] != "convt_attend_query"] == [
        (f"convt_{n}", 1) for n in ("rms_norm", "cache_write", "cache_read", "attend", "q4_matvec")]
    plan = C.get_plan((1, 4, 8, 8), (4, 4, 3, 3))
    monkeypatch.setattr(C, "_lib", two_devices)
    del two_devices.calls[:]
    plan.forward(t(1, 4, 8, 8, dtype=torch.float32), t(4, 4, 3, 3, dtype=torch.float32), y=t(*plan.out_shape, dtype=torch.float32),
                 workspace=t(1 << 16, dtype=torch.uint8))
    plan.backward_data(t(*plan.out_shape, dtype=torch.float32), t(4, 4, 3, 3, dtype=torch.float32), dx=t(1, 4, 8, 8, dtype=torch.float32),
                       workspace=t(1 << 16, dtype=torch.uint8))
    assert two_devices.calls == [("convt_forward", 1), ("convt_backward_data", 1)] and two_devices.now == 0


def test_slots_of_positions_outside_the_table():
    """A position before the first token or past the table has no slot; it took another page's place, or none on the device."""
    table = torch.tensor([[3, 0], [7, -1]], dtype=torch.int32)
    got = C.cache_slots(table, torch.tensor([0, 0, 0, 0, 1, 0]), torch.tensor([-1, -16, -17, 32, 31, 31]), 16)
    assert got.dtype == torch.int64 and got[:4].tolist() == [-1] * 4 and got[4] < 0 and got[5] == 15
    assert C.cache_slots(table, torch.tensor([1]), torch.tensor([10 ** 9]), 16).tolist() == [-1]
    assert C.cache_slots(table, torch.tensor(1), torch.arange(-2, 3), 16).tolist() == [-1, -1, 112, 113, 114]
    assert C.cache_slots(table[:, :0], torch.tensor([0, 1]), torch.tensor([0, 5]), 16).tolist() == [-1, -1]
    assert C.cache_slots(table, torch.tensor([0, 1], dtype=torch.int64), torch.tensor([17, 1], dtype=torch.int32), 16).tolist() == [1, 113]
