"""Which stream the binding's allocations belong to when a call runs on a
stream of the caller's choice (CPU: torch and the library are stand-ins that
keep account).

A tensor that a call allocates is written on that call's stream. Torch hands
out memory that a stream freed to that stream's next allocation at once, while
work queued there may still use it, so the call's tensors have to be allocated
on the stream that the call runs on, and the caller's current stream recorded
as a reader of those that are returned."""

import contextlib

import pytest

from packed_attention_qk_b200 import pqk


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return isinstance(other, Stream) and other.cuda_stream == self.cuda_stream


class Tensor:
    next_ptr = 0x10000

    def __init__(self, dtype, shape, strides=None, owner=None):
        self.dtype, self.shape, self.owner, self.readers = dtype, tuple(shape), owner, []
        if strides is None:
            strides, n = [], 1
            for d in reversed(self.shape):
                strides.insert(0, n)
                n *= d
        self._strides = tuple(strides)
        self.device = "cuda:0"
        self.ptr, Tensor.next_ptr = Tensor.next_ptr, Tensor.next_ptr + 0x10000
        self.is_cuda = True

    def dim(self):
        return len(self.shape)

    def stride(self, d=None):
        return self._strides if d is None else self._strides[d]

    def get_device(self):
        return 0

    def is_contiguous(self):
        n = 1
        for d, s in zip(reversed(self.shape), reversed(self._strides)):
            if s != n:
                return False
            n *= d
        return True

    def numel(self):
        n = 1
        for d in self.shape:
            n *= d
        return n

    def element_size(self):
        return 2 if self.dtype == "bfloat16" else 4 if self.dtype in ("float32", "int32") else 1

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def data_ptr(self):
        return self.ptr

    def record_stream(self, s):
        self.readers.append(s)

    def __getitem__(self, index):
        """A range of a vector, or the first columns of a matrix's rows."""
        if isinstance(index, slice):
            shape = (len(range(*index.indices(self.shape[0]))),)
        else:
            shape = (self.shape[0], index[1].stop)
        t = Tensor(self.dtype, shape, self._strides, self.owner)
        t.ptr, t.readers = self.ptr, self.readers
        return t


class Torch:
    """As much of torch as the binding's calls touch."""

    Tensor = Tensor
    bfloat16, float32, int32, int8, uint8 = "bfloat16", "float32", "int32", "int8", "uint8"

    def __init__(self):
        self.current = self.main = Stream(0)
        self.made = []
        outer = self

        class C:
            _cuda_getDevice = staticmethod(lambda: 0)
            _cuda_getCurrentRawStream = staticmethod(lambda dev: outer.current.cuda_stream)

        class Cuda:
            ExternalStream = staticmethod(lambda handle: Stream(handle if handle else 0xDEAD))
            default_stream = staticmethod(lambda: outer.main)
            current_stream = staticmethod(lambda: outer.current)
            current_device = staticmethod(lambda: 0)

            @staticmethod
            @contextlib.contextmanager
            def stream(s):
                before, outer.current = outer.current, s
                yield
                outer.current = before

        self._C, self.cuda = C, Cuda

    def empty_strided(self, shape, strides, dtype, device):
        self.made.append(Tensor(dtype, shape, strides, owner=self.current))
        return self.made[-1]

    def empty(self, shape, dtype, device):
        return self.empty_strided((shape,) if isinstance(shape, int) else shape, None, dtype, device)

    def empty_like(self, t):
        return self.empty_strided(t.shape, None, t.dtype, t.device)


class Library:
    """Every call succeeds; what it was given is kept."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 256 if name.endswith("workspace_size") else 0
        return call


@pytest.fixture
def fake(monkeypatch):
    torch, library = Torch(), Library()
    monkeypatch.setattr(pqk, "_torch", torch)
    monkeypatch.setitem(__import__("sys").modules, "torch", torch)
    monkeypatch.setattr(pqk, "lib", lambda: library)
    pqk.varlen_cross_attn_workspace_size.cache_clear()
    yield torch, library
    pqk.varlen_cross_attn_workspace_size.cache_clear()


def _bf(*shape):
    return Tensor("bfloat16", shape)


def _cu(n):
    return Tensor("int32", (n,))


I8_CALLS = {
    "norm_modulate_i8": lambda s: pqk.norm_modulate_i8(_bf(4, 64), stream=s)[1:],
    "quantize_i8": lambda s: pqk.quantize_i8(_bf(4, 40), stream=s),
    "linear_i8_gated_residual": lambda s: pqk.linear_i8_gated_residual(
        Tensor("int8", (4, 64)), Tensor("float32", (4,)), Tensor("int8", (32, 64)), Tensor("float32", (32,)), stream=s),
    "linear_i8_swiglu": lambda s: pqk.linear_i8_swiglu(
        Tensor("int8", (4, 64)), Tensor("float32", (4,)), Tensor("int8", (32, 64)), Tensor("float32", (32,)), stream=s),
    "varlen_cross_attn_fwd": lambda s: pqk.varlen_cross_attn_fwd(
        _bf(4, 2, 64), _bf(5, 2, 64), _bf(5, 2, 64), _cu(3), _cu(3), want_lse=True, stream=s),
}


def _check(fake, call, stream, handle):
    torch, library = fake
    returned = call(stream)
    returned = returned if isinstance(returned, tuple) else (returned,)
    assert torch.made and library.calls[-1][1][-1] == handle
    assert all(t.owner.cuda_stream == handle for t in torch.made)
    assert torch.current is torch.main
    if handle != torch.main.cuda_stream:
        returned_ptrs = {t.ptr for t in returned if isinstance(t, Tensor)}
        for t in torch.made:
            assert t.ptr not in returned_ptrs or torch.main in t.readers


@pytest.mark.parametrize("name", I8_CALLS)
def test_new_tensors_belong_to_the_calls_stream(fake, name):
    _check(fake, I8_CALLS[name], Stream(7), 7)


@pytest.mark.parametrize("name", I8_CALLS)
def test_raw_handles_and_the_default_stream(fake, name):
    _check(fake, I8_CALLS[name], 9, 9)
    fake[0].made.clear()
    _check(fake, I8_CALLS[name], 0, 0)
    fake[0].made.clear()
    _check(fake, I8_CALLS[name], None, 0)


def test_the_callers_tensors_are_recorded_on_the_calls_stream(fake):
    x8, scales = Tensor("int8", (4, 64)), Tensor("float32", (4,))
    pqk.quantize_i8(_bf(4, 64), x8=x8, scales=scales, stream=Stream(7))
    assert not fake[0].made and Stream(7) in x8.readers and Stream(7) in scales.readers


def _f32(*shape):
    return Tensor("float32", shape)


def _u8(*shape):
    return Tensor("uint8", shape)


CALLS = {
    "qk_norm_rope_e4m3": lambda s: pqk.qk_norm_rope_e4m3(_bf(4, 2, 128), _bf(4, 2, 128), _bf(128), _bf(128), _cu(4),
                                                         stream=s),
    "varlen_attn_fwd": lambda s: pqk.varlen_attn_fwd(_bf(4, 2, 64), _bf(4, 2, 64), _bf(4, 2, 64), _cu(3),
                                                     want_lse=True, stream=s),
    "varlen_attn_fwd_skip": lambda s: pqk.varlen_attn_fwd_skip(_bf(4, 2, 64), _bf(4, 2, 64), _bf(4, 2, 64), _cu(3),
                                                               8.0, want_lse=True, stream=s),
    "quantize_qk_e4m3": lambda s: pqk.quantize_qk_e4m3(_bf(4, 2, 128), _bf(4, 2, 128), stream=s),
    "varlen_attn_fwd_fp8qk": lambda s: pqk.varlen_attn_fwd_fp8qk(
        _u8(4, 2, 128), _u8(4, 2, 128), _bf(4, 2, 128), _f32(4), _cu(3), want_lse=True, stream=s),
    "quantize_e4m3": lambda s: pqk.quantize_e4m3(_bf(4, 2, 128), stream=s),
    "varlen_attn_fwd_fp8": lambda s: pqk.varlen_attn_fwd_fp8(
        _u8(4, 2, 128), _u8(4, 2, 128), _u8(4, 2, 128), _f32(6), _cu(3), want_lse=True, stream=s),
    "varlen_attn_fwd_noalloc": lambda s: pqk.varlen_attn_fwd_noalloc(
        _bf(4, 2, 64), _bf(4, 2, 64), _bf(4, 2, 64), _cu(3), want_lse=True, stream=s),
    "modulate_swiglu": lambda s: pqk.modulate_swiglu(_bf(4, 64), _f32(2, 64), _f32(2, 64), _cu(3), gate=_bf(4, 64),
                                                     up=_bf(4, 64), stream=s),
    "linear_gated_residual": lambda s: pqk.linear_gated_residual(_bf(4, 64), _bf(32, 64), stream=s),
    "linear_swiglu": lambda s: pqk.linear_swiglu(_bf(4, 64), _bf(32, 64), stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_new_tensors_of_the_bf16_and_fp8_calls(fake, name):
    for stream, handle in ((Stream(7), 7), (9, 9), (0, 0), (None, 0)):
        fake[0].made.clear()
        _check(fake, CALLS[name], stream, handle)
