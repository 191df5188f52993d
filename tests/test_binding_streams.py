"""Who owns what the binding allocates for a call on another stream than the current one.  Scratch
must come from that stream's pool (what is freed at return is handed out again only behind the
call's kernels), outputs too, and those are marked as used on the caller's stream.  A fake of torch
and of the library: no GPU, no kernel."""
import contextlib
import ctypes
import types

import pytest

from weight_only_bit_q4_gb300 import q4lin


class Stream:
    def __init__(self, n):
        self.cuda_stream = n


class Tensor:
    is_cuda = True

    def __init__(self, shape, dtype, stream=None, cuda=True):
        self.shape, self.dtype, self.stream, self.used_on, self.is_cuda = tuple(shape), dtype, stream, [], cuda
        self.device = types.SimpleNamespace(index=0, type="cuda")

    def is_contiguous(self):
        return True

    def element_size(self):
        return {"u8": 1, "f32": 4, "i32": 4}.get(self.dtype, 2)

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

    def record_stream(self, s):
        self.used_on.append(s)

    def pin_memory(self):
        return self


class FakeTorch(types.SimpleNamespace):
    def __init__(self):
        super().__init__(uint8="u8", bfloat16="bf", float32="f32", int32="i32", int16="i16")
        self.main, self.made = Stream(1), []
        self.now = self.main
        self.cuda = types.SimpleNamespace(current_stream=lambda device=None: self.now, stream=self.under)
        self._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: self.now.cuda_stream)

    @contextlib.contextmanager
    def under(self, s):
        before, self.now = self.now, s
        yield
        self.now = before

    def empty(self, *shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        t = Tensor(shape, dtype, self.now, cuda=device is not None)
        if device is not None:
            self.made.append(t)
        return t


class FakeLib:
    def __getattr__(self, name):
        def f(*args):
            if name.endswith("workspace_bytes"):
                return 4096
            self.stream = args[-1].value if isinstance(args[-1], ctypes.c_void_p) else args[-1]
            return 0
        return f


T, K, N, L, R, E, F, H, k = 2, 128, 64, 3, 8, 4, 128, 128, 2


def bf(*s):
    return Tensor(s, "bf")


CALLS = {
    "linear": lambda s: q4lin.linear(Tensor((N, K // 2), "u8"), bf(N, K // 64), bf(T, K), stream=s),
    "linear_add": lambda s: q4lin.linear_add(Tensor((N, K // 2), "u8"), bf(N, K // 64), bf(T, K), bf(T, N), stream=s),
    "linear_qtype": lambda s: q4lin.linear_qtype("w8g32", (Tensor((N, K), "u8"),), bf(N, K // 32), bf(T, K), stream=s),
    "linear_swiglu": lambda s: q4lin.linear_swiglu(Tensor((N, K // 2), "u8"), bf(N, K // 64), bf(T, K), stream=s),
    "linear_pair": lambda s: q4lin.linear_pair(Tensor((N, K // 2), "u8"), bf(N, K // 64), Tensor((N, K // 2), "u8"),
                                               bf(N, K // 64), bf(T, K), stream=s),
    "linear_host": lambda s: q4lin.linear_host(Tensor((N, K // 2), "u8"), bf(N, K // 64), Tensor((T, K), "bf", cuda=False),
                                               stream=s),
    "linear_lora": lambda s: q4lin.linear_lora(Tensor((N, K // 2), "u8"), bf(N, K // 64), bf(T, K), bf(L, R, K), bf(L, N, R),
                                               Tensor((T,), "i32"), stream=s),
    "moe_router": lambda s: q4lin.moe_router(bf(T, H), bf(E, H), k, stream=s),
    "moe_experts": lambda s: q4lin.moe_experts(bf(T, H), Tensor((T, k), "i32"), Tensor((T, k), "f32"), *planes(), stream=s),
    "moe": lambda s: q4lin.moe(bf(T, H), bf(E, H), *planes(), k, stream=s),
    "qk_norm_rope": lambda s: q4lin.qk_norm_rope(bf(T, 64), bf(T, 32), bf(32), bf(32), Tensor((16, 32), "f32"),
                                                 Tensor((T,), "i32"), stream=s),
}


def planes():
    return (Tensor((E, 2 * F, H // 2), "u8"), bf(E, 2 * F, H // 64), Tensor((E, H, F // 2), "u8"), bf(E, H, F // 64))


@pytest.fixture
def fake(monkeypatch):
    torch, lib = FakeTorch(), FakeLib()
    monkeypatch.setattr(q4lin, "_torch", torch)
    monkeypatch.setitem(__import__("sys").modules, "torch", torch)
    monkeypatch.setattr(q4lin, "load", lambda path=None: lib)
    return torch, lib


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_another_stream_owns_its_tensors_there(fake, name):
    torch, lib = fake
    side = Stream(7)
    out = CALLS[name](side)
    outs = [o for o in (out if isinstance(out, tuple) else (out,)) if o.is_cuda]
    assert lib.stream == 7 and torch.now is torch.main
    assert torch.made and all(t.stream is side for t in torch.made)
    assert all(t.used_on == [torch.main] for t in outs)
    assert all(any(t is o for o in outs) or not t.used_on for t in torch.made)   # scratch goes back to its stream alone


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_the_current_stream(fake, name):
    torch, lib = fake
    CALLS[name](None)
    assert lib.stream == 1 and all(t.stream is torch.main and not t.used_on for t in torch.made)
    torch.made.clear()
    CALLS[name](torch.main)   # named, but the current one
    assert lib.stream == 1 and all(t.stream is torch.main and not t.used_on for t in torch.made)
