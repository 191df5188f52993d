"""The cache attention's workspace is as large as the device of the call wants it, whatever device is current and
whatever sizes were asked for before.  A fake of torch and of the library: no GPU, no kernel."""
import contextlib
import types

import pytest

from weight_only_bit_q4_gb300 import q4lin

NEED = {0: 4096, 1: 8192}      # bytes per device


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.index = tuple(shape), dtype, index
        self.device = types.SimpleNamespace(index=index, type="cuda")

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return True

    def element_size(self):
        return {"u8": 1, "i32": 4}.get(self.dtype, 2)

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self):
        st, n = [], 1
        for s in reversed(self.shape):
            st.insert(0, n)
            n *= s
        return tuple(st)

    def data_ptr(self):
        return 256


class FakeTorch(types.SimpleNamespace):
    def __init__(self):
        super().__init__(uint8="u8", bfloat16="bf", int32="i32")
        self.index, self.made = 0, []
        self.cuda = types.SimpleNamespace(device=self.on)
        self._C = types.SimpleNamespace(_cuda_getDevice=lambda: self.index, _cuda_getCurrentRawStream=lambda i: 1)

    @contextlib.contextmanager
    def on(self, index):
        before, self.index = self.index, index
        yield
        self.index = before

    def empty(self, shape, dtype=None, device=None):
        t = Tensor((shape,) if isinstance(shape, int) else shape, dtype, device.index)
        self.made.append(t)
        return t


class FakeLib:
    def __init__(self, torch):
        self.torch, self.ran_on = torch, []

    def q4lin_kv4_page_bytes(self, D):
        return 4352

    def q4lin_kv4_workspace_bytes(self, *sizes):
        return NEED[self.torch.index]

    def q4lin_kv4_attention(self, *args):
        self.ran_on.append(self.torch.index)
        return 0


@pytest.fixture
def fake(monkeypatch):
    torch = FakeTorch()
    lib = FakeLib(torch)
    monkeypatch.setattr(q4lin, "_torch", torch)
    monkeypatch.setattr(q4lin, "load", lambda path=None: lib)
    monkeypatch.setattr(q4lin, "_KV_NEED", {})
    monkeypatch.setattr(q4lin, "_PAGE_BYTES", {})
    return torch, lib


def call(index, **kw):
    return q4lin.kv4_attention(Tensor((2, 4, 64), "bf", index), Tensor((3, 2, 4352), "u8", index), Tensor((2, 5), "i32", index),
                               Tensor((2,), "i32", index), **kw)


def scratch(torch):
    return [t.numel() for t in torch.made if t.dtype == "u8"]


@pytest.mark.parametrize("order", [(0, 1), (1, 0), (1, 1, 0, 1)])
@pytest.mark.parametrize("current", [0, 1])
def test_the_workspace_is_the_calls_devices(fake, order, current):
    torch, lib = fake
    torch.index = current
    for index in order:
        torch.made.clear()
        call(index)
        assert scratch(torch) == [NEED[index]]
    assert lib.ran_on == list(order) and torch.index == current


def test_a_workspace_of_another_devices_size_is_refused(fake):
    torch, _ = fake
    call(0, workspace=Tensor((NEED[0],), "u8", 0))
    with pytest.raises(ValueError):
        call(1, workspace=Tensor((NEED[0],), "u8", 1))
    call(1, workspace=Tensor((NEED[1],), "u8", 1))


def test_the_query_answers_for_the_current_or_a_named_device(fake):
    torch, _ = fake
    sizes = (2, 1, 4, 2, 64, 5)
    for current in (0, 1, 0):
        torch.index = current
        assert q4lin.kv4_workspace_bytes(*sizes) == NEED[current]
        assert [q4lin.kv4_workspace_bytes(*sizes, device=i) for i in (0, 1)] == [NEED[0], NEED[1]]
    assert torch.index == 0
