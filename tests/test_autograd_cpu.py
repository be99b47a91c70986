"""The operators record nothing for autograd, so a tensor that requires a gradient is
refused where gradients are on; without them, and inside a torch.autograd.Function, it
is a tensor like any other.  On the CPU: an accepted call stops at the device check."""
import pytest
import torch

from block_scaled_precision_amd import moe_mx as m

T, H, E, K, N = 4, 128, 6, 2, 16
BF16, I32, U8 = torch.bfloat16, torch.int32, torch.uint8


def _f(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "moe_permute": (dict(x=_f(T, H), sorted_assign=_f(T * K, dtype=I32), expert_offsets=_f(E + 1, dtype=I32), k=K),
                    dict(rows=_f(T * K, H))),
    "moe_permute_backward": (dict(drows=_f(T * K, H), row_of=_f(T, K, dtype=I32)), dict(dx=_f(T, H))),
    "moe_unpermute": (dict(rows=_f(T * K, H), row_of=_f(T, K, dtype=I32), topk_w=_f(T, K), residual=_f(T, H)),
                      dict(y=_f(T, H))),
    "moe_unpermute_backward": (dict(dy=_f(T, H), rows=_f(T * K, H), row_of=_f(T, K, dtype=I32), topk_w=_f(T, K)),
                               dict(drows=_f(T * K, H), dw=_f(T, K))),
    "moe_route_backward": (dict(topk_ids=_f(T, K, dtype=I32), topk_w=_f(T, K), dw=_f(T, K), num_experts=E),
                           dict(dlogits=_f(T, E))),
    "mx_linear": (dict(a=_f(T, H, dtype=BF16), w=_f(N, H // 2, dtype=U8), w_scale=_f(N, H // 32, dtype=U8), fmt="e2m1",
                       act="bf16", bias=_f(N), mul=_f(T, N, dtype=BF16), residual=_f(T, N, dtype=BF16)),
                  dict(out=_f(T, N, dtype=BF16))),
}
TENSORS = [(op, name) for op, (given, outs) in CALLS.items() for name, t in {**given, **outs}.items()
           if isinstance(t, torch.Tensor) and t.is_floating_point()]


def _arguments(op, name):
    given, outs = CALLS[op]
    kw = dict(given, **{k: v for k, v in outs.items() if k == name})
    kw[name] = kw[name].clone().requires_grad_()
    return kw


@pytest.mark.parametrize("op,name", TENSORS)
def test_a_tensor_that_requires_a_gradient_is_refused(op, name):
    kw = _arguments(op, name)
    with pytest.raises(ValueError, match=f"^{name} requires a gradient, which {op} does not"):
        getattr(m, op)(**kw)
    with pytest.raises(ValueError, match=f"^{name} requires a gradient"):
        m.OpCall(getattr(m, op), **kw)


@pytest.mark.parametrize("op,name", TENSORS)
def test_without_gradients_it_goes_on(op, name):
    kw = _arguments(op, name)
    for mode in (torch.no_grad, torch.inference_mode):
        with mode(), pytest.raises(ValueError, match="GPU"):
            getattr(m, op)(**kw)

    class Own(torch.autograd.Function):
        @staticmethod
        def forward(ctx, t):
            return getattr(m, op)(**{**kw, name: t})

    with pytest.raises(ValueError, match="GPU"):
        Own.apply(kw[name])
