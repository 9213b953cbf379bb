"""The routed experts' bindings without a GPU: CPU tensors that say they are on a GPU, and stand-ins for the calls."""
import pytest

torch = pytest.importorskip("torch")

import moe_shared_expert_gb300 as mse
from moe_shared_expert_gb300 import _build, routed


class On:
    """A CPU tensor that gives `index` for its CUDA device."""

    def __init__(self, t, index):
        self.t, self.index = t, index
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture
def calls(monkeypatch):
    """The operators' calls: names of those that were reached."""
    _build.build()
    routed._load()
    reached = []

    def take(name):
        return lambda *a: reached.append(name) or 0

    for name in ("route", "linear", "matmul", "experts"):
        monkeypatch.setattr(routed, "_call_" + name, take(name))

    class C:
        fp8_block_quantise = staticmethod(take("quantise"))

    monkeypatch.setattr(routed, "_C", C)
    monkeypatch.setattr(routed, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(routed, "_current", lambda: 0, raising=False)
    monkeypatch.setattr(routed, "_empty", lambda stream, shape, dtype, device: On(torch.empty(shape, dtype=dtype), device.index))
    return reached


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def e4m3(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


OPERATORS = {
    "route": (mse.moe_route, dict(logits=torch.zeros(3, 8), top_k=2, bias=torch.zeros(8),
                                  ids=torch.zeros(3, 2, dtype=torch.int32), weights=torch.zeros(3, 2))),
    "quantise": (mse.fp8_block_quantise, dict(x=bf16(3, 64))),
    "matmul": (mse.fp8_block_matmul, dict(xq=e4m3(3, 64), xs=torch.zeros(3, 1), wq=e4m3(5, 64), ws=torch.zeros(1, 1), out=bf16(3, 5))),
    "linear": (mse.fp8_block_linear, dict(x=bf16(3, 64), wq=e4m3(5, 64), ws=torch.zeros(1, 1), y=bf16(3, 5), workspace=e4m3(1 << 12))),
    "experts": (mse.moe_experts_forward, dict(x=bf16(3, 64), ids=torch.zeros(3, 2, dtype=torch.int32), weights=torch.zeros(3, 2),
                                              w_gate_up=e4m3(4, 32, 64), s_gate_up=torch.zeros(4, 2, 1), w_down=e4m3(4, 64, 16),
                                              s_down=torch.zeros(4, 1, 1), shared=bf16(3, 64), y=bf16(3, 64), workspace=e4m3(1 << 20))),
}
TENSORS = [(op, name) for op, (_, a) in OPERATORS.items() for name, v in a.items() if isinstance(v, torch.Tensor)]


def arguments(op, index=0, **other):
    f, a = OPERATORS[op]
    return f, {n: On(v, index) if isinstance(v, torch.Tensor) else v for n, v in {**a, **other}.items()}


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_of_the_current_device_are_taken(calls, op):
    f, a = arguments(op)
    f(**a)
    assert calls == [op]


@pytest.mark.parametrize("op", OPERATORS)
def test_tensors_of_another_device_than_the_current_one_are_refused(calls, op):
    f, a = arguments(op, index=1)
    with pytest.raises(ValueError, match="cuda:1"):
        f(**a)
    assert calls == []


@pytest.mark.parametrize("op,name", TENSORS)
def test_a_tensor_of_another_device_or_of_the_cpu_is_refused(calls, op, name):
    f, a = arguments(op)
    on = a[name]
    for wrong in (On(on.t, 1), on.t):
        with pytest.raises(ValueError, match=name):
            f(**{**a, name: wrong})
    assert calls == []


@pytest.mark.parametrize("op", ["linear", "experts"])
def test_a_workspace_with_holes_is_refused(calls, op):
    f, a = arguments(op)
    for wrong in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 21, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            f(**{**a, "workspace": On(wrong, 0)})
    assert calls == []


class FakeCuda:
    """torch.cuda of one device: streams, and which of them is current."""

    class Stream:
        def __init__(self, handle):
            self.cuda_stream = handle

    def __init__(self):
        self.now = self.Stream(0)
        self.default = self.now

    def current_stream(self, device=None):
        return self.now

    def default_stream(self, device=None):
        return self.default

    def ExternalStream(self, handle, device=None):
        assert handle != 0, "a handle of 0 makes a new stream"
        return self.Stream(handle)

    def stream(self, s):
        import contextlib

        @contextlib.contextmanager
        def entered():
            before, self.now = self.now, s
            yield
            self.now = before
        return entered()


@pytest.fixture
def made(monkeypatch):
    """(tensors, cuda): what the bindings allocate, with the stream that was current and the streams it was recorded on."""
    routed._load()
    cuda, tensors = FakeCuda(), []

    class Made:
        def __init__(self, shape):
            self.shape, self.allocated_on, self.recorded = shape, cuda.now.cuda_stream, []
            tensors.append(self)

        def record_stream(self, s):
            self.recorded.append(s.cuda_stream)

    class Torch:
        uint8 = torch.uint8
        empty = staticmethod(lambda shape, dtype=None, device=None: Made(shape))

    Torch.cuda = cuda
    monkeypatch.setattr(routed, "torch", Torch)
    return tensors, cuda


@pytest.mark.parametrize("as_handle", [False, True])
def test_memory_for_another_stream_is_that_streams(made, as_handle):
    # a block that the current stream has let go may still be read and written by its kernels: what another stream
    # fills comes from that stream's own blocks, and is not taken again before the current stream, too, is done with it
    tensors, cuda = made
    side = 77 if as_handle else cuda.Stream(77)
    routed._empty(side, (3, 4), torch.bfloat16, "cuda:0")
    assert tensors[-1].allocated_on == 77 and tensors[-1].recorded == [0] and cuda.now.cuda_stream == 0
    cuda.now = cuda.Stream(5)
    routed._empty(0 if as_handle else cuda.default, (3, 4), torch.bfloat16, "cuda:0")
    assert tensors[-1].allocated_on == 0 and tensors[-1].recorded == [5]
    routed._empty(None, (3, 4), torch.bfloat16, "cuda:0")
    assert tensors[-1].allocated_on == 5 and tensors[-1].recorded == []


@pytest.mark.parametrize("op", ["linear", "experts"])
def test_a_workspace_for_another_stream_is_that_streams(calls, monkeypatch, op):
    asked = []
    monkeypatch.setattr(routed, "_empty", lambda stream, shape, dtype, device: asked.append((stream, shape, dtype)) or On(e4m3(shape), 0))
    f, a = arguments(op)
    f(**{**a, "workspace": None}, stream=77)
    need = mse.fp8_linear_workspace_bytes(3, 5, 64) if op == "linear" else mse.moe_workspace_bytes(3, 2, 4, 64, 16)
    assert asked == [(77, need, torch.uint8)] and calls == [op]
