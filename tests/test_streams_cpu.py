"""Memory of tensors that a call uses on another stream than their own: the binding
tells the allocator.  On the CPU with stand-ins for tensors, streams and the launch."""
import contextlib

import pytest
import torch

from block_scaled_precision_amd import moe_mx as m


class Memory:
    """A tensor as the allocator sees it: the streams that were recorded."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream.cuda_stream)


class Device:
    index = 0


DEVICE = Device()


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, DEVICE


@pytest.fixture
def cuda(monkeypatch):
    """The current stream is cuda["stream"], under capture if cuda["capturing"]."""
    state = {"stream": Stream(1), "capturing": False}
    monkeypatch.setattr(m.torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m.torch.cuda, "current_stream", lambda device=None: state["stream"])
    monkeypatch.setattr(m.torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(m.torch._C, "_cuda_getCurrentRawStream", lambda index: state["stream"].cuda_stream, raising=False)
    return state


def _plan(result, keep, status=m.MOE_OK):
    plan = m._Plan("moe_route_backward", (0, 0, 0, 1, 8, 2, 0), result, DEVICE, keep)
    launched = []
    plan.fn = lambda *args: launched.append(args[-1]) or status
    return plan, launched


def test_prepared_calls_record_every_stream_once(cuda):
    out, out2, given, ws = (Memory() for _ in range(4))
    plan, launched = _plan((out, out2), (given, None, ws))
    for handle in (1, 1, 2, 1, 2):
        cuda["stream"] = Stream(handle)
        assert plan.launch(None, prepared=True) == (out, out2)
    assert launched == [1, 1, 2, 1, 2]
    assert all(t.streams == [1, 2] for t in (out, out2, given, ws))


def test_a_stream_argument_records_inputs_and_outputs(cuda):
    out, given = Memory(), Memory()
    plan, launched = _plan(out, (given,))
    assert plan.launch(Stream(7)) is out
    assert launched == [7] and out.streams == given.streams == [7]


def test_calls_on_the_current_stream_leave_the_caller_s_tensors_alone(cuda):
    out, given = Memory(), Memory()
    plan, _ = _plan(out, (given,))
    plan.launch(None)
    assert out.streams == given.streams == []


def test_a_record_under_capture_does_not_last(cuda):
    out = Memory()
    plan, _ = _plan(out, ())
    cuda["capturing"] = True
    plan.launch(None, prepared=True)
    plan.launch(None, prepared=True)
    assert out.streams == [1, 1]
    cuda["capturing"] = False
    plan.launch(None, prepared=True)
    plan.launch(None, prepared=True)
    assert out.streams == [1, 1, 1]


def test_a_failed_launch_records_nothing(cuda):
    out = Memory()
    plan, _ = _plan(out, (), status=m.MOE_ERR_HIP)
    with pytest.raises(m.MoeError):
        plan.launch(None, prepared=True)
    assert out.streams == []


@pytest.fixture
def entry_points(cuda, monkeypatch):
    """The entry points on CPU tensors, launching nothing: what they record, as
    {address: handles}, and the launches' streams."""
    recorded, launched = {}, []

    class Library:
        def __getattr__(self, name):
            if name.endswith("_bytes"):
                return lambda *args: 64
            return lambda *args: launched.append(getattr(args[-1], "value", args[-1])) or m.MOE_OK

    monkeypatch.setattr(m, "lib", Library)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(m, "_dev", lambda *ts: None)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, stream: recorded.setdefault(t.data_ptr(), []).append(stream.cuda_stream))
    return recorded, launched


BF16, U8 = torch.bfloat16, torch.uint8
T, H, I, E, K = 4, 64, 32, 4, 2


def _layer():
    u8 = lambda *shape: torch.zeros(shape, dtype=U8)
    weights = m.MoeWeights(u8(E, 2 * I, H // 2), u8(E, 2 * I, H // 32), u8(E, H, I // 2), u8(E, H, I // 32), "e2m1")
    given = (torch.zeros((T, H), dtype=BF16), torch.zeros((T, E)))
    return m.make_problem(T, H, I, E, K, "e2m1", "bf16"), weights, *given


@pytest.mark.parametrize("name", ["mx_quantize", "moe_route", "mx_gemm", "moe_fused"])
def test_entry_points_with_a_stream_argument(entry_points, monkeypatch, name):
    """Inputs, outputs and the workspace that the call allocates for itself, from the
    stream's memory and for the current one to read."""
    recorded, launched = entry_points
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(empty(*a, **kw)) or made[-1])
    a, codes, scales = torch.zeros((T, 128), dtype=BF16), torch.zeros((8, 64), dtype=U8), torch.zeros((8, 4), dtype=U8)
    problem, weights, x, logits = _layer()
    given = {"mx_quantize": (a, "e4m3"), "moe_route": (logits, K), "mx_gemm": (a, codes, scales, "e2m1"),
             "moe_fused": (problem, x, weights, logits)}[name]
    getattr(m, name)(*given)
    assert recorded == {}
    made.clear()
    getattr(m, name)(*given, stream=Stream(5))
    assert launched == [1, 5]
    tensors = [t for t in given if isinstance(t, torch.Tensor)]
    if name == "moe_fused":
        tensors += [weights.w1, weights.w1_scale, weights.w2, weights.w2_scale]
    assert all(recorded.get(t.data_ptr()) == [5] for t in tensors)
    assert made and all(recorded.get(t.data_ptr()) == [1, 5] for t in made)


def test_prepared_layer_records_every_stream_once(cuda, entry_points):
    recorded, launched = entry_points
    problem, weights, x, logits = _layer()
    call = m.FusedCall(problem, x, weights, logits)
    for handle in (1, 2, 2, 1):
        cuda["stream"] = Stream(handle)
        y = call()
    assert launched == [1, 2, 2, 1]
    workspace = call._keep[6]
    assert all(recorded.get(t.data_ptr()) == [1, 2] for t in (x, logits, y, workspace, weights.w1, weights.w2_scale))
