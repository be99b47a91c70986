"""Pins for the dispatch oracle (CPU only): a hand-written example, the routing
oracle's permutation, and torch's automatic differentiation in float64."""
import numpy as np
import pytest
import torch

from oracle import dispatch as od
from oracle import routing as orouting


def test_hand_example():
    ids = np.array([[2, 0], [0, 1], [2, 1]])
    assert od.row_of(ids, 3).tolist() == [[4, 0], [1, 2], [5, 3]]
    assert od.row_of(ids, 3, 1, 1).tolist() == [[-1, -1], [-1, 0], [-1, 1]]
    x = np.array([[1.0], [2.0], [3.0]])
    assert od.permute(x, od.row_of(ids, 3), np.zeros((7, 1))).ravel().tolist() == [1, 2, 2, 3, 1, 3, 0]
    w = np.array([[0.25, 0.75], [0.5, 0.5], [1.0, 0.0]])
    rows = np.arange(6.0)[:, None]
    y, size = od.unpermute(rows, od.row_of(ids, 3), w, np.array([[-1.0], [0.0], [0.0]]))
    assert y.ravel().tolist() == [0.0, 1.5, 5.0] and size.ravel().tolist() == [2.0, 1.5, 5.0]


@pytest.mark.parametrize("lo,n", [(0, 9), (3, 4), (8, 1)])
def test_rows_match_the_routing_oracle(lo, n):
    rng = np.random.default_rng(1)
    ids, _ = orouting.topk_route(rng.standard_normal((20, 9)).astype(np.float32), 3)
    _, offsets, order = orouting.permute(ids, 9, lo, n)
    r = od.row_of(ids, 9, lo, n)
    assert [r.ravel()[a] for a in order] == list(range(offsets[-1]))
    assert np.count_nonzero(r >= 0) == offsets[-1]


@pytest.mark.parametrize("lo,n", [(0, 6), (2, 3)])
def test_gradients_match_autograd(lo, n):
    rng = np.random.default_rng(2)
    T, k, E, H = 7, 3, 6, 5
    logits = torch.from_numpy(rng.standard_normal((T, E)))
    ids, _ = orouting.topk_route(logits.numpy().astype(np.float32), k)
    r = od.row_of(ids, E, lo, n)
    here = torch.from_numpy(r >= 0)
    idx = torch.from_numpy(np.maximum(r, 0))
    x = torch.from_numpy(rng.standard_normal((T, H))).requires_grad_()
    logits.requires_grad_()
    gain = torch.from_numpy(rng.standard_normal((T * k, H)))
    dy = rng.standard_normal((T, H))
    w = torch.softmax(torch.gather(logits, 1, torch.from_numpy(ids).long()), 1)
    w.retain_grad()
    token = np.zeros(T * k, dtype=np.int64)
    for t, j in zip(*np.nonzero(r >= 0)):
        token[r[t, j]] = t
    rows = x[torch.from_numpy(token)] * gain
    rows.retain_grad()
    y = (rows[idx] * (w * here)[..., None]).sum(1)
    y.backward(torch.from_numpy(dy))
    drows, dw, _ = od.unpermute_backward(dy, rows.detach().numpy(), r, w.detach().numpy(), np.zeros((T * k, H)))
    np.testing.assert_allclose(drows, rows.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(dw, w.grad.numpy(), atol=1e-13)
    dx, _ = od.unpermute(drows * gain.numpy(), r)
    np.testing.assert_allclose(dx, x.grad.numpy(), atol=1e-13)
    np.testing.assert_allclose(od.route_backward(ids, w.detach().numpy(), dw, E), logits.grad.numpy(), atol=1e-13)
