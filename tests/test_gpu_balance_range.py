"""moe_balance and its gradient where the logits are far from 0, up to the largest and the lowest
of the type, against the formulas in 64 bits.

A probability is off by the rounding of its argument, |x - lse| half steps of fp32, by that of
the exponential and by the relative error of the row's sum, sum_j p_j (|x_j - lse| + 28); a
factor that is common to a row's exponentials, as lse's own rounding makes one, is none of it.
The other steps as oracle/balance.py counts them."""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from tests.conftest import has_gpu
from tests.helpers import print_flush
from tests.test_gpu_balance import E32, F32, _np

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

LOWEST, LARGEST = torch.finfo(F32).min, torch.finfo(F32).max


def _reference(x, ids, dloss):
    """(losses, gradient, bound of the gradient in half steps) of one sequence of counted tokens."""
    T, E = x.shape
    m = x.max(1, keepdims=True)
    e = np.exp(x - m)
    p, lse = e / e.sum(1, keepdims=True), m + np.log(e.sum(1, keepdims=True))
    far = np.where(p > 0, np.abs(x - m) + 2 * np.log(E), 0.0)  # lse, rounded, is at most 2 log E above max
    f = np.bincount(ids.ravel(), minlength=E) / ids.size
    row = (p * (far + 28)).sum(1, keepdims=True)
    rel = far + row + 16
    a, b = dloss[0] * E / T, dloss[1] * 2 / T
    dot, dot_size = (p * f).sum(1, keepdims=True), (p * f * (rel + 24)).sum(1, keepdims=True)
    out = a * p * (f - dot) + b * lse * p
    size = abs(a) * p * ((rel + 8) * (f + dot) + dot_size) + abs(b) * p * (np.abs(lse) * (rel + 10) + row + 2 * np.log(E))
    with np.errstate(over="ignore"):
        return (E * (f * p.mean(0)).sum(), (lse ** 2).mean()), out, size + 2 * np.abs(out)


def _check(x, k, dloss):
    from block_scaled_precision_amd import moe_mx as m
    T, E = x.shape
    ids = torch.topk(x, k, dim=1).indices.int()
    loss, counts, tokens, lse = m.moe_balance(x.cuda(), ids.cuda())
    assert tokens.tolist() == [T, T, 1]
    d = torch.tensor(dloss, dtype=F32)
    g = _np(m.moe_balance_backward(d.cuda(), x.cuda(), counts, tokens, lse, k))
    ref, want, size = _reference(_np(x), ids.numpy(), _np(d))
    assert not np.isnan(g).any()
    # (results below 2^-126, of sums of E terms and products with lse)
    tiny = 2.0 ** -126 * (E + 4) * (abs(dloss[0]) * E + 2 * abs(dloss[1]) * (np.abs(_np(lse)).max() + 1) + 1)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(g - want) <= size * E32 + tiny) & ~((np.abs(want) > LARGEST) & (g == np.copysign(np.inf, want)))
    assert not bad.any(), (np.argwhere(bad)[:3], g[bad][:3], want[bad][:3], (size * E32)[bad][:3])
    # P is off by |x - max| (20 at most where it counts), the row's sum (50) and its additions (80
    # with the product); lse by the row's sum, 2 |lse| and 2 log E, its square's sum by 64 more
    assert abs(loss[0].item() / ref[0] - 1) <= 160 * E32
    if ref[1] < LARGEST:
        assert abs(loss[1].item() / ref[1] - 1) <= 200 * E32
    else:
        assert loss[1].item() == float("inf")


@pytest.mark.parametrize("T,E,k", [(5, 7, 2), (60, 64, 4), (300, 130, 3), (400, 384, 8)])
@pytest.mark.parametrize("base", [0.0, 1e3, -1e5, 1e7, -3e8, 2e9, 1e20])
def test_logits_with_a_common_offset(T, E, k, base):
    print_flush(f"moe_balance T={T} E={E} offset {base}")
    x = gen.normal((T, E), T, 1, std=2.0) + torch.tensor(base)
    _check(x, k, (0.7, 0.0))
    _check(x, k, (0.7, -1.3))


@pytest.mark.parametrize("T,E,k", [(60, 64, 4), (300, 130, 3)])
def test_rows_of_the_lowest_and_the_largest_value(T, E, k):
    """All logits alike, or a few above others at the lowest value: the softmax is uniform over
    those, whatever their size."""
    x = gen.normal((T, E), T, 2)
    x[3] = LOWEST
    x[4] = LARGEST
    x[5, 2:] = LOWEST
    x[6], x[6, :5] = LOWEST, LARGEST
    x[7], x[7, 1] = 1e30, -1e30
    x[8], x[8, ::2] = -1e4, -1e4 + 1
    _check(x, k, (0.7, 0.0))


@pytest.mark.parametrize("dloss", [(0.7, 1.0), (0.0, -65536.0), (3.0, 2.0 ** -20)])
@pytest.mark.parametrize("E", [8, 33, 200])
def test_z_terms_at_the_end_of_the_range(E, dloss):
    """2 lse / n past fp32's largest number, where the term itself is not, or is 0."""
    rows = [torch.full((E,), LOWEST), torch.full((E,), LARGEST), torch.full((E,), LOWEST), torch.full((E,), -3e38),
            torch.arange(E) * 1e36]
    rows[2][1::2] = -1e38
    rows[3][E // 2:] = LOWEST
    for r in rows:
        _check(r.float()[None], 2, dloss)
    _check(torch.stack([r.float() for r in rows]), 2, dloss)
