"""The dispatch operators inside torch.autograd.Functions, as a training step uses them:
gradients of a routed layer against autograd of the same formulas in 64 bits.

With e = 2^-24: the router's weights are off by at most 8 e of their value, a product
of two fp32 numbers by e, a sum of n terms in fp32 by n e times the sum of magnitudes.
"""
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

E32 = 2.0 ** -24


def _functions(m):
    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, k):
            ids, w, off, order = m.moe_route(logits, k)
            ctx.save_for_backward(ids, w)
            ctx.experts = logits.shape[1]
            ctx.mark_non_differentiable(ids, off, order)
            return ids, w, off, order

        @staticmethod
        def backward(ctx, _ids, dw, _off, _order):
            ids, w = ctx.saved_tensors
            return m.moe_route_backward(ids, w, dw.contiguous(), ctx.experts), None

    class Permute(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, order, off, k):
            rows, row_of = m.moe_permute(x, order, off, k)
            ctx.save_for_backward(row_of)
            ctx.mark_non_differentiable(row_of)
            return rows, row_of

        @staticmethod
        def backward(ctx, drows, _):
            return m.moe_permute_backward(drows, *ctx.saved_tensors), None, None, None

    class Unpermute(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rows, row_of, w, residual):
            ctx.save_for_backward(rows, row_of, w)
            return m.moe_unpermute(rows, row_of, w, residual=residual)

        @staticmethod
        def backward(ctx, dy):
            drows, dw = m.moe_unpermute_backward(dy, *ctx.saved_tensors)
            return drows, None, dw, dy

    return Route, Permute, Unpermute


@pytest.mark.parametrize("T,H,E,k", [(1, 64, 4, 2), (50, 264, 12, 3), (300, 1031, 9, 4)])
def test_gradients_of_a_routed_layer(T, H, E, k):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"autograd T={T} H={H} E={E} k={k}")
    Route, Permute, Unpermute = _functions(m)
    x, logits = (gen.normal(s, 60, i).cuda().requires_grad_() for i, s in ((1, (T, H)), (2, (T, E))))
    gain = gen.normal((E, H), 60, 3).cuda().requires_grad_()
    dy = gen.normal((T, H), 60, 4).cuda()
    ids, w, off, order = Route.apply(logits, k)
    rows, row_of = Permute.apply(x, order, off, k)
    expert = torch.repeat_interleave(torch.arange(E, device="cuda"), (off[1:] - off[:-1]).long())
    y = Unpermute.apply(rows * gain[expert], row_of, w, x)
    y.backward(dy)

    x64, l64, g64 = (t.detach().double().requires_grad_() for t in (x, logits, gain))
    w64 = torch.softmax(l64.gather(1, ids.long()), 1)
    picked = g64[ids.long()]  # [T, k, H]
    y64 = x64 + (w64[..., None] * picked * x64[:, None]).sum(1)
    y64.backward(dy.double())

    def within(got, ref, bound, what):
        worst = ((got.double() - ref).abs() / bound.clamp(min=1e-300)).max().item()
        assert worst <= 1.0, f"{what}: worst ratio {worst:.3f}"

    with torch.no_grad():
        d = dy.double().abs()
        terms = w64[..., None] * picked.abs()  # of y and of dx
        within(y, y64, (k + 12) * E32 * (x64.abs() + (terms * x64.abs()[:, None]).sum(1)) + E32 * y64.abs(), "y")
        within(x.grad, x64.grad, (k + 13) * E32 * d * (1 + terms.sum(1)), "dx")
        # a row's part of its expert's gradient, summed over the expert's rows
        part = (w64[..., None] * (d * x64.abs())[:, None]).view(T * k, H)
        size = torch.zeros((E, H), dtype=torch.float64, device="cuda").index_add_(0, ids.view(-1).long(), part)
        within(gain.grad, g64.grad, (T + 12) * E32 * size, "dgain")
        dw = (dy.double()[:, None] * picked * x64[:, None]).sum(2)
        off_by = (H + 2) * E32 * (d[:, None] * picked.abs() * x64.abs()[:, None]).sum(2)
        own = w64 * ((dw.abs() + (w64 * dw.abs()).sum(1, keepdim=True)) * (k + 4 + 24) * E32 + off_by
                     + (w64 * off_by).sum(1, keepdim=True))
        bound = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), own)
        within(logits.grad, l64.grad, bound, "dlogits")
        assert not logits.grad[bound == 0].any()


def test_a_graph_that_would_be_lost_is_refused():
    from block_scaled_precision_amd import moe_mx as m
    ids, w, off, order = m.moe_route(gen.normal((4, 6), 61, 1).cuda(), 2)
    x = gen.normal((4, 32), 61, 2).cuda().requires_grad_()
    with pytest.raises(ValueError, match="x requires a gradient"):
        m.moe_permute(x, order, off, 2)
    with torch.no_grad():
        rows, row_of = m.moe_permute(x, order, off, 2)
    assert torch.equal(rows, x.detach()[order.long() // 2]) and not rows.requires_grad
