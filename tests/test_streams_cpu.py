"""Memory of tensors that a call uses on another stream than their own: the binding
tells the allocator.  On the CPU with stand-ins for tensors, streams and the launch."""
import pytest

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


def test_a_capture_is_no_use_and_the_next_call_still_records(cuda):
    out = Memory()
    plan, _ = _plan(out, ())
    cuda["capturing"] = True
    plan.launch(None, prepared=True)
    assert out.streams == []
    cuda["capturing"] = False
    plan.launch(None, prepared=True)
    assert out.streams == [1]


def test_a_failed_launch_records_nothing(cuda):
    out = Memory()
    plan, _ = _plan(out, (), status=m.MOE_ERR_HIP)
    with pytest.raises(m.MoeError):
        plan.launch(None, prepared=True)
    assert out.streams == []
