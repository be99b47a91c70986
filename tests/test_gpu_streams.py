"""Calls on another stream than the one their tensors come from: memory that a call
still running on it uses is not handed out again.  Every case keeps that stream busy
with a wait that ends by itself, drops everything the call used, and allocates the
same sizes at once."""
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

BF16 = torch.bfloat16
CYCLES = 20_000_000  # 8 ms and more, whichever clock the wait counts
T, H, E, K = 600, 2048, 8, 2


def _operators(m):
    """name -> (operator, inputs made anew on the current stream)"""
    ids, w, off, order = m.moe_route(gen.normal((T, E), 50, 30).cuda(), K)
    x = gen.normal((T, H), 50, 31).to(BF16)
    rows, row_of = m.moe_permute(x.cuda(), order, off, K)
    codes, scales = m.mx_quantize(gen.normal((1024, H), 50, 32, std=0.02).cuda(), "e2m1")
    torch.cuda.synchronize()

    def c(*ts):
        return tuple(t.clone() if isinstance(t, torch.Tensor) else t for t in ts)

    return {
        "permute": (m.moe_permute, lambda: c(x.cuda(), order, off, K)),
        "permute_backward": (m.moe_permute_backward, lambda: c(rows, row_of)),
        "unpermute": (m.moe_unpermute, lambda: c(rows, row_of, w)),
        "unpermute_backward": (m.moe_unpermute_backward, lambda: c(x.cuda(), rows, row_of, w)),
        "route_backward": (m.moe_route_backward, lambda: c(ids, w, w, E)),
        "linear": (m.mx_linear, lambda: (*c(x.cuda(), codes, scales), "e2m1", "mxfp8")),
    }


def _ranges(*ts):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in ts if isinstance(t, torch.Tensor)]


def _free_of(used):
    """Allocates as much as `used` several times over and returns it; none of it may
    lie in `used`."""
    new = [torch.empty(hi - lo, dtype=torch.uint8, device="cuda") for lo, hi in used for _ in range(3)]
    for a, b in _ranges(*new):
        for lo, hi in used:
            assert b <= lo or hi <= a, "memory of a running call was handed out"
    return new


NAMES = ["permute", "permute_backward", "unpermute", "unpermute_backward", "route_backward", "linear"]


@pytest.mark.parametrize("name", NAMES)
def test_prepared_call_dropped_while_it_runs(name):
    """Built on one stream, called on another and dropped: outputs, inputs and the
    workspace stay until the call is through."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"streams: prepared {name}")
    op, make = _operators(m)[name]
    side = torch.cuda.Stream()
    args = make()
    call = m.OpCall(op, *args)
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
        out = call()
    outputs = out if isinstance(out, tuple) else (out,)
    used = _ranges(*args, *outputs, *call._plan.keep)
    assert not side.query()
    del args, call, out, outputs
    new = _free_of(used)
    torch.cuda.synchronize()
    del new


@pytest.mark.parametrize("name", NAMES)
def test_stream_argument_with_inputs_dropped(name):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"streams: argument {name}")
    op, make = _operators(m)[name]
    side = torch.cuda.Stream()
    want = op(*make())
    args = make()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    out = op(*args, stream=side)
    used = _ranges(*args)
    assert not side.query()
    del args
    for t in _free_of(used):
        t.fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    for got, ref in zip(out if isinstance(out, tuple) else (out,), want if isinstance(want, tuple) else (want,)):
        assert torch.equal(got, ref)


def test_prepared_call_captured_then_called_and_dropped():
    """A capture neither fails nor stands for a call that ran."""
    from block_scaled_precision_amd import moe_mx as m
    op, make = _operators(m)["linear"]
    args = make()
    want = op(*args)
    call = m.OpCall(op, *args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    out.zero_()
    assert torch.equal(call(), want)
    del graph, call, out
    torch.cuda.synchronize()
    assert torch.equal(op(*args), want)
