"""Pins for the router-balance oracle (CPU only): hand-worked cases, invariants, torch's
automatic differentiation in float64, and differences."""
import numpy as np
import pytest
import torch

from oracle import balance as ob


def _case(T, E, k, offsets, seed=0, masked=True):
    rng = np.random.default_rng(seed)
    logits = rng.standard_normal((T, E)) * 2
    logits[rng.random((T, E)) < 0.1] = -np.inf
    logits[T // 2] = -np.inf  # a token with nothing to choose
    ids = np.argsort(-logits, axis=1)[:, :k]
    mask = rng.random(T) < 0.8 if masked else None
    return logits, ids, mask


def test_even_routing_costs_one():
    """Equal logits and every expert chosen equally often: balance 1, lse log E."""
    E = 6
    ids = np.array([[t % E, (t + 1) % E] for t in range(12)])
    loss, counts, tokens, lse, _, _ = ob.balance(np.zeros((12, E)), ids, 1, [0, 12])
    assert np.allclose(loss, [1.0, np.log(E) ** 2]) and (counts == 4).all() and tokens.tolist() == [12, 12, 1]
    assert np.allclose(lse, np.log(E))


def test_one_expert_for_all_costs_as_many_as_there_are():
    logits = np.full((5, 4), -np.inf)
    logits[:, 2] = 1.0
    loss, counts, _, lse, _, _ = ob.balance(logits, np.full((5, 1), 2), 1, [0, 5])
    assert np.allclose(loss, [4.0, 1.0]) and counts.tolist() == [[0, 0, 5, 0]] and np.allclose(lse, 1.0)


def test_hand_example():
    """Two sequences of one and two tokens, an empty one, a masked token and one outside."""
    a = np.log([[1.0, 3.0], [1.0, 1.0], [2.0, 2.0], [7.0, 1.0], [5.0, 5.0]])
    ids = np.array([[1], [0], [1], [0], [0]])
    loss, counts, tokens, lse, _, _ = ob.balance(a, ids, 3, [0, 1, 1, 4], np.array([1, 1, 1, 0, 1]))
    assert counts.tolist() == [[0, 1], [0, 0], [1, 1]] and tokens.tolist() == [1, 0, 2, 3, 2]
    # first: 2 * (0 * 1/4 + 1 * 3/4); last: 2 * (1/2 * 1/2 + 1/2 * 1/2)
    assert np.allclose(loss[0], (1.5 + 1.0) / 2)
    assert np.allclose(loss[1], (np.log(4) ** 2 + np.log(2) ** 2 + np.log(4) ** 2) / 3)
    assert np.allclose(lse[:3], np.log([4, 2, 4])) and (lse[3:] == -np.inf).all()


@pytest.mark.parametrize("offsets", [[0, 13], [0, 4, 4, 9], [2, 3, 11]])
def test_gradient_matches_autograd(offsets):
    logits, ids, mask = _case(13, 7, 3, offsets)
    S = len(offsets) - 1
    loss, counts, tokens, _, _, _ = ob.balance(logits, ids, S, offsets, mask)
    d = np.array([0.7, -1.3])
    add = np.random.default_rng(1).standard_normal(logits.shape)
    got, _ = ob.balance_backward(d, logits, counts, tokens, 3, offsets, mask, add)
    x = torch.from_numpy(logits).requires_grad_()
    seq = ob.counted(logits, offsets, mask)
    value = torch.zeros((), dtype=torch.float64)
    for t in np.flatnonzero(seq >= 0):
        finite = torch.from_numpy(np.flatnonzero(logits[t] > -np.inf))
        p, f = torch.softmax(x[t, finite], 0), torch.from_numpy(counts[seq[t]] / (3 * tokens[seq[t]]))[finite]
        value = value + d[0] * 7 / tokens[-1] * (f * p).sum() / tokens[seq[t]]
        value = value + d[1] * torch.logsumexp(x[t, finite], 0) ** 2 / tokens[-2]
    assert np.allclose(value.item(), d @ loss)
    value.backward()
    np.testing.assert_allclose(got - add, x.grad.numpy(), atol=1e-13)


def test_gradient_matches_differences():
    logits, ids, _ = _case(6, 5, 2, [0, 6], masked=False)
    logits[logits == -np.inf] = -1.0
    offsets, d, h = [0, 2, 6], np.array([1.0, 0.5]), 1e-5
    _, counts, tokens, _, _, _ = ob.balance(logits, ids, 2, offsets)
    grad, _ = ob.balance_backward(d, logits, counts, tokens, 2, offsets)
    for t in range(6):
        for e in range(5):
            up, down = logits.copy(), logits.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = d @ (ob.balance(up, ids, 2, offsets)[0] - ob.balance(down, ids, 2, offsets)[0]) / (2 * h)
            assert abs(diff - grad[t, e]) < 1e-8


def test_what_does_not_count_changes_nothing():
    logits, ids, mask = _case(20, 6, 2, [0, 17])
    ref = ob.balance(logits, ids, 1, [0, 17], mask)
    other = logits.copy()
    other[~mask] = np.nan
    other[17:] = np.nan
    for a, b in zip(ref, ob.balance(other, ids, 1, [0, 17], mask)):
        assert np.array_equal(a, b)
    grad, _ = ob.balance_backward(np.ones(2), logits, ref[1], ref[2], 2, [0, 17], mask)
    seq = ob.counted(logits, [0, 17], mask)
    assert (grad[seq < 0] == 0).all() and np.isfinite(grad).all()
    # a token's probabilities sum to one, so the balance part of its gradient sums to zero
    part, _ = ob.balance_backward(np.array([1.0, 0.0]), logits, ref[1], ref[2], 2, [0, 17], mask)
    assert np.abs(part.sum(1)).max() < 1e-14
