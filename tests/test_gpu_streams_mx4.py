"""The balance and MXFP4 operators on another stream than the one their tensors come from, and
the losses inside a torch.autograd.Function."""
import numpy as np
import pytest
import torch

import tests.test_gpu_streams as streams
from block_scaled_precision_amd import inputs as gen
from oracle import balance as ob
from tests.conftest import has_gpu
from tests.test_gpu_balance import E32, _case, _np

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

T, H, E, K = streams.T, streams.H, streams.E, streams.K


def _operators(m):
    """name -> (operator, inputs made anew on the current stream)"""
    logits = gen.normal((T, E), 60, 30)
    ids, *_ = m.moe_route(logits.cuda(), K)
    so = torch.tensor([0, 100, 100, 350, T - 50], dtype=torch.int32)
    mask = torch.arange(T) % 7 != 0
    loss, counts, tokens, lse = m.moe_balance(logits.cuda(), ids, mask.cuda(), so.cuda())
    x = gen.normal((T, H), 60, 31).to(torch.bfloat16)
    signs = torch.where(gen.random_bytes((32,), 60, 32) < 128, -1.0, 1.0)
    random = gen.random_bytes((T, H), 60, 33)
    w = m.mx4_quantize(gen.normal((1024, H), 60, 34, std=0.02).cuda())
    wg = m.mx4_quantize(gen.normal((4, 1024, H), 60, 35, std=0.02).cuda())
    off = torch.tensor([0, 1, 300, 300, T], dtype=torch.int32)
    torch.cuda.synchronize()

    def linear(a, codes, scales, offsets=None, **kw):
        return m.mx4_linear(a, codes, scales, expert_offsets=offsets, **kw)

    def plan(a, codes, scales, offsets=None, **kw):
        return m._PLANNERS[m.mx4_linear](a, codes, scales, expert_offsets=offsets, **kw)
    m._PLANNERS[linear] = plan
    return {
        "balance": (m.moe_balance, lambda: (logits.cuda(), ids.clone(), mask.cuda(), so.cuda())),
        "balance_backward": (m.moe_balance_backward, lambda: (torch.ones(2, device="cuda"), logits.cuda(), counts.clone(),
                                                              tokens.clone(), lse.clone(), K, so.cuda(), logits.cuda())),
        "quantize4": (m.mx4_quantize, lambda: (x.cuda(), False, signs.cuda(), random.cuda())),
        "quantize4_transposed": (m.mx4_quantize, lambda: (x.cuda(), True, signs.cuda(), random.cuda())),
        "dequantize4": (m.mx4_dequantize, lambda: (w[0].clone(), w[1].clone())),
        "linear4": (linear, lambda: (x.cuda(), w[0].clone(), w[1].clone())),
        "linear4_grouped": (linear, lambda: (x.cuda(), wg[0].clone(), wg[1].clone(), off.cuda())),
    }


NAMES = ["balance", "balance_backward", "quantize4", "quantize4_transposed", "dequantize4", "linear4", "linear4_grouped"]


@pytest.fixture
def operators(monkeypatch):
    from block_scaled_precision_amd import moe_mx as m
    monkeypatch.setattr(m, "_PLANNERS", dict(m._PLANNERS))
    monkeypatch.setattr(streams, "_operators", _operators)


@pytest.mark.parametrize("name", NAMES)
def test_prepared_call_dropped_while_it_runs(name, operators):
    streams.test_prepared_call_dropped_while_it_runs(name)


@pytest.mark.parametrize("name", NAMES)
def test_stream_argument_with_inputs_dropped(name, operators):
    streams.test_stream_argument_with_inputs_dropped(name)


def _balance_function(m):
    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids, mask, so):
            loss, counts, tokens, lse = m.moe_balance(logits, ids, mask, so)
            ctx.save_for_backward(logits, counts, tokens, lse, so)
            ctx.k = ids.shape[1]
            ctx.mark_non_differentiable(counts, tokens, lse)
            return loss, counts, tokens, lse

        @staticmethod
        def backward(ctx, dloss, *_):
            logits, counts, tokens, lse, so = ctx.saved_tensors
            return m.moe_balance_backward(dloss.contiguous(), logits, counts, tokens, lse, ctx.k, so), None, None, None
    return Balance


@pytest.mark.parametrize("T,E,k,S", [(90, 16, 2, 3), (500, 96, 4, 5)])
def test_losses_in_a_graph_of_autograd(T, E, k, S):
    """The gradient of a weighted sum of both losses (a broadcast gradient among them) against
    autograd of the formulas in 64 bits; half steps as oracle/balance.py counts them."""
    from block_scaled_precision_amd import moe_mx as m
    logits, ids, mask, off = _case(T, E, k, S, 12, masked=True)
    so = torch.from_numpy(off).int().cuda()
    for weights in (None, torch.tensor([0.25, 0.5])):
        x = logits.cuda().requires_grad_()
        loss, counts, tokens, _ = _balance_function(m).apply(x, ids.cuda(), mask.cuda(), so)
        (loss.sum() if weights is None else (loss * weights.cuda()).sum()).backward()
        d = np.ones(2) if weights is None else _np(weights)
        y = logits.double().requires_grad_()
        balance, z, used = 0.0, 0.0, 0
        for s in range(S):
            rows = torch.arange(off[s], off[s + 1])[mask[off[s]:off[s + 1]]]
            if not len(rows):
                continue
            used += 1
            c = torch.bincount(ids[rows].flatten().long(), minlength=E)
            assert torch.equal(c.int(), counts[s].cpu())
            balance = balance + E * (c.double() / (k * len(rows)) * torch.softmax(y[rows], 1).mean(0)).sum()
            z = z + (torch.logsumexp(y[rows], 1) ** 2).sum()
        total = d[0] * balance / used + d[1] * z / tokens[S].item()
        total.backward()
        _, size = ob.balance_backward(d, _np(logits), counts.cpu().numpy(), tokens.cpu().numpy(), k, off, mask.numpy())
        # (1e-13: the reference's own steps in 64 bits)
        assert (np.abs(_np(x.grad) - y.grad.numpy()) <= size * E32 + 1e-13).all()
