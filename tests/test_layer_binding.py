"""What the layer operators' binding refuses before it calls the library: stand-ins for
tensors on several GPUs, and a stand-in for the library that notes every call (no GPU)."""

import ctypes as C

import pytest

import block_quant_gb300 as bq

P = 1 << 20  # an address that nothing reads


class Tensor:
    """What the binding reads off a torch tensor."""

    SIZE = {"bf16": 2, "f32": 4, "u8": 1, "i32": 4, "i64": 8, "odd": 8}

    def __init__(self, dtype, *shape, gpu=0, at=P, contiguous=True):
        self.dtype, self.shape, self.gpu, self.at, self.whole = dtype, tuple(shape), gpu, at, contiguous

    def stride(self):
        s = [1]
        for k in reversed(self.shape[1:]):
            s.insert(0, s[0] * k)
        return tuple(s)

    def is_contiguous(self):
        return self.whole

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return self.at

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def element_size(self):
        return self.SIZE[self.dtype]

    @property
    def nbytes(self):
        return self.numel() * self.element_size()


class Library:
    """bq_call's stand-in: the packed calls that reached it."""

    KINDS = {"bf16": 0, "f32": 1, "u8": 2, "i32": 32, "i64": 64}

    def __init__(self):
        self.calls, self.current = [], 0
        self.entry = C.CFUNCTYPE(C.c_int, C.c_int, C.c_void_p)(self._call)

    def _call(self, op, words):
        self.calls.append((op, [C.cast(words, C.POINTER(C.c_int64))[i] for i in range(8)]))
        return 0

    def bind(self, module, fill=None):
        module.bind(C.cast(self.entry, C.c_void_p).value, dict(self.KINDS), fill or (lambda dtype: None),
                    lambda: self.current)


@pytest.fixture
def library(monkeypatch):
    from block_quant_gb300 import build

    build.build()
    module = bq._layer()
    fake = Library()
    fake.bind(module)
    yield fake
    bq._calls = None  # the next call binds the library again
    bq._layer()


def embed(gpu=0, **change):
    a = dict(table=Tensor("bf16", 10, 16, gpu=gpu), ids=Tensor("i64", 4, gpu=gpu), out=Tensor("bf16", 4, 16, gpu=gpu))
    a.update(change)
    bq.embed(**a, stream=0)


def test_calls_reach_the_library(library):
    embed()
    assert [op for op, _ in library.calls] == [0]
    assert library.calls[0][1][0] == P and library.calls[0][1][3:5] == [10, 16]


def test_tensors_on_several_gpus_are_refused(library):
    for name, t in (("ids", Tensor("i64", 4, gpu=1)), ("out", Tensor("bf16", 4, 16, gpu=1)), ("out", Tensor("bf16", 4, 16, gpu=-1))):
        with pytest.raises(bq.BQError, match="GPU"):
            embed(**{name: t})
    assert not library.calls


def test_a_call_made_while_another_reads_its_tensors(library):
    """Reading an unknown type runs Python code, in which another call may be made (from this
    thread, or by a switch to another): the outer call's GPU stays its own."""
    def fill(dtype):
        if nested:
            embed(gpu=1)
        return 64

    module = bq._layer()
    library.current = 1
    for nested in (False, True):
        library.bind(module, fill)
        library.calls.clear()
        with pytest.raises(bq.BQError, match="another GPU"):
            embed(ids=Tensor("odd", 4, gpu=1), out=Tensor("bf16", 4, 16, gpu=1))  # the table is on GPU 0
        assert len(library.calls) == int(nested)  # the inner one alone


WS = Tensor("u8", 1 << 20)
X, W, F8, S = Tensor("bf16", 4, 16), Tensor("bf16", 16), Tensor("u8", 4, 16), Tensor("f32", 1, 4)
WITH_WORKSPACE = {
    "embed_grad": lambda ws: bq.embed_grad(X, Tensor("i64", 4), Tensor("bf16", 10, 16), ws, stream=0),
    "rmsnorm_grad": lambda ws: bq.rmsnorm_grad(X, X, W, Tensor("f32", 4), X, W, ws, stream=0),
    "linear_fp8": lambda ws: bq.linear_fp8(F8, S, Tensor("u8", 8, 16), Tensor("f32", 1), Tensor("bf16", 4, 8), ws, stream=0),
    "linear_fp8_dx": lambda ws: bq.linear_fp8_dx(Tensor("bf16", 4, 8), Tensor("u8", 8, 16), Tensor("f32", 1), X, ws, stream=0),
    "linear_fp8_dw": lambda ws: bq.linear_fp8_dw(Tensor("bf16", 4, 8), F8, S, Tensor("bf16", 8, 16), ws, stream=0),
}


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspaces(library, name):
    """A workspace in host memory, on another GPU, with gaps, or that is no tensor, never
    reaches the library; one of any type on the call's GPU does."""
    call = WITH_WORKSPACE[name]
    for ws in (WS, Tensor("f32", 3, 5, 7)):
        call(ws)
    assert len(library.calls) == 2
    for ws in (Tensor("u8", 1 << 20, gpu=-1), Tensor("u8", 1 << 20, gpu=1), Tensor("u8", 1 << 20, contiguous=False), None,
               P, "ws"):
        with pytest.raises(bq.BQError) as e:
            call(ws)
        assert e.value.code == bq.BQ_EINVAL
    assert len(library.calls) == 2


def test_the_checked_workspace_is_on_a_gpu():
    import torch

    for ws in (torch.zeros(256, dtype=torch.uint8), None, P):
        with pytest.raises(bq.BQError) as e:
            bq.linear_check(ws, stream=0)
        assert e.value.code == bq.BQ_EINVAL


def test_the_current_device_is_the_tensors(library):
    """A call runs on the current device's stream, by its sizes: tensors elsewhere are refused."""
    with pytest.raises(bq.BQError, match="current device") as e:
        embed(gpu=1)
    assert e.value.code == bq.BQ_EINVAL and not library.calls
    library.current = 1
    embed(gpu=1)
    assert len(library.calls) == 1
    for call in WITH_WORKSPACE.values():
        with pytest.raises(bq.BQError, match="current device"):
            call(WS)
    with pytest.raises(bq.BQError, match="current device"):
        bq.rmsnorm(X, W, 1e-5, y=X, stream=0)
    with pytest.raises(bq.BQError, match="current device"):
        bq.quant_rows_fp8(X, F8, S, stream=0)
    with pytest.raises(bq.BQError, match="current device"):
        bq.linear_check(WS, stream=0)
    assert len(library.calls) == 1
