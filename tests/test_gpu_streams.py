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


def _entry_points(m):
    """name -> (entry point, inputs made anew on the current stream)"""
    x, logits = gen.normal((T, H), 51, 31).to(BF16), gen.normal((T, E), 51, 30)
    codes, scales = m.mx_quantize(gen.normal((1024, H), 51, 32, std=0.02).cuda(), "e2m1")
    w1, s1 = m.mx_quantize(gen.normal((E, 2 * 512, H), 51, 33, std=0.02).cuda(), "e2m1")
    w2, s2 = m.mx_quantize(gen.normal((E, H, 512), 51, 34, std=0.02).cuda(), "e2m1")
    problem = m.make_problem(T, H, 512, E, K, "e2m1", "mxfp8")
    torch.cuda.synchronize()
    return {
        "quantize": (m.mx_quantize, lambda: (x.cuda(), "e4m3")),
        "route": (m.moe_route, lambda: (logits.cuda(), K)),
        "gemm": (m.mx_gemm, lambda: (x.cuda(), codes.clone(), scales.clone(), "e2m1")),
        "fused": (m.moe_fused, lambda: (problem, x.cuda(), m.MoeWeights(w1, s1, w2, s2, "e2m1"), logits.cuda())),
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


@pytest.mark.parametrize("name", NAMES + ["quantize", "route", "gemm", "fused"])
def test_stream_argument_with_inputs_dropped(name):
    """Inputs, and workspaces that the call allocates and drops itself: what comes in
    their place is filled at once, and the results are those of an undisturbed call."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"streams: argument {name}")
    op, make = {**_operators(m), **_entry_points(m)}[name]
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
    for size in (1 << 16, 1 << 18, 1 << 20, 3 << 20, 8 << 20):
        torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xFF)
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


def test_prepared_layer_dropped_while_it_runs():
    from block_scaled_precision_amd import moe_mx as m
    make = _entry_points(m)["fused"][1]
    args = make()
    call = m.FusedCall(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
        y = call()
    used = _ranges(args[1], args[3], y, call._keep[6])
    assert not side.query()
    del args, call, y
    new = _free_of(used)
    torch.cuda.synchronize()
    del new


def test_stream_argument_under_capture():
    """A side stream forked inside a capture: inputs dropped there are not reused by
    what the capture allocates next."""
    from block_scaled_precision_amd import moe_mx as m
    op, make = _operators(m)["linear"]
    base = make()
    want = op(base[0] * 2, *base[1:])
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        a = base[0] * 2
        side.wait_stream(main)
        out = op(a, *base[1:], stream=side)
        del a
        other = base[0] * 3  # of a's size, while the side stream reads a
        main.wait_stream(side)
    for _ in range(4):
        out.zero_()
        other.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, base[0] * 3)
