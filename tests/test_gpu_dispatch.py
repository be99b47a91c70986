"""Dispatch operators on the GPU against the float64 oracle.

Routing comes from moe_route, so each case is the chain a user runs.  Bounds,
with u = half a unit in the last place of the output type (2^-8 bf16, 2^-24
fp32) and e = 2^-24 for every fp32 operation:
* moving rows is exact;
* a sum of n terms in fp32 in any order is off by at most n e times the sum of
  its terms' magnitudes (n counts the products' own roundings), and its one
  output rounding by u times the value;
* a single product, rounded to fp32 and then to the output type, by (e + u)
  times the value (for fp32 outputs it is one rounding).
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from oracle import dispatch as od
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

E32 = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _assert_within(got, ref, bound, what):
    d = np.abs(_np(got) - ref)
    bad = np.flatnonzero(~(d <= bound))
    assert bad.size == 0, f"{what}: {bad.size} of {d.size} out of bounds, worst {np.nanmax(d - bound):.3e}"


def _routed(T, E, k, seed=0):
    from block_scaled_precision_amd import moe_mx as m
    logits = gen.normal((T, E), seed, 30).cuda()
    return m.moe_route(logits, k)


def _rand(shape, seed, dtype):
    return gen.normal(shape, seed, 31).to(dtype).cuda()


# (T, H, E, k, local_offset, local_count): one token, odd and tiny rows, more
# slots than are in flight at once, rows of many pieces, shards down to one expert
CASES = [
    (1, 7168, 384, 8, 0, 0), (1, 1, 1, 1, 0, 0), (5, 333, 7, 3, 0, 0), (3, 8, 4, 4, 1, 2), (64, 1024, 32, 8, 0, 0),
    (64, 1024, 32, 8, 16, 16), (257, 72, 20, 11, 0, 0), (33, 4104, 64, 17, 7, 1), (130, 520, 512, 6, 100, 300),
    (2, 64, 16, 2, 15, 1), (11, 16896, 8, 3, 0, 0), (3, 4100, 16, 12, 2, 9), (256, 1032, 8, 2, 0, 0),
    (300, 1544, 32, 11, 0, 0), (9000, 1000, 8, 2, 0, 0), (4500, 2000, 8, 2, 0, 0),
    (2100, 4100, 16, 9, 3, 9), (8200, 1031, 16, 2, 0, 0), (520, 4099, 16, 4, 2, 11),
]


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,H,E,k,lo,n", CASES)
def test_operators_match_the_oracle(T, H, E, k, lo, n, dtype):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"dispatch T={T} H={H} E={E} k={k} local={lo}+{n} {dtype}")
    u = _half_step(dtype)
    ids, w, off, order = _routed(T, E, k)
    x = _rand((T, H), 1, dtype)
    ref_of = od.row_of(ids.cpu().numpy(), E, lo, n or E)
    sentinel = 77.0
    rows = torch.full((T * k, H), sentinel, dtype=dtype, device="cuda")
    out, row_of = m.moe_permute(x, order, off, k, local_offset=lo, local_count=n, rows=rows)
    torch.cuda.synchronize()
    assert out is rows and np.array_equal(row_of.cpu().numpy(), ref_of)
    assert np.array_equal(_np(rows), od.permute(_np(x), ref_of, np.full((T * k, H), sentinel)))

    # rows no assignment names hold NaN, and so do the weights of absent ones:
    # neither may reach an output
    g = _rand((T * k, H), 2, dtype)
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[row_of[row_of >= 0].long()] = True
    g[~named] = float("nan")
    wn = torch.where(row_of >= 0, w, torch.full_like(w, float("nan")))
    g64, w64 = np.where(named.cpu().numpy()[:, None], _np(g), 0.0), np.where(ref_of >= 0, _np(w), 0.0)

    ref, size = od.unpermute(g64, ref_of)
    _assert_within(m.moe_permute_backward(g, row_of), ref, u * np.abs(ref) + (1 + u) * k * E32 * size, "dx")
    res = _rand((T, H), 3, dtype)
    for r in (None, res):
        ref, size = od.unpermute(g64, ref_of, w64, None if r is None else _np(r))
        bound = u * np.abs(ref) + (1 + u) * (k + 1) * E32 * size
        _assert_within(m.moe_unpermute(g, row_of, wn, residual=r), ref, bound, "y")
    y = res.clone()  # in place over the residual
    assert m.moe_unpermute(g, row_of, wn, residual=y, y=y) is y
    _assert_within(y, ref, bound, "y in place")

    dy = _rand((T, H), 4, dtype)
    drows = torch.full((T * k, H), sentinel, dtype=dtype, device="cuda")
    _, dw = m.moe_unpermute_backward(dy, g, row_of, wn, drows=drows)
    ref, dw_ref, dw_size = od.unpermute_backward(_np(dy), g64, ref_of, w64, np.full((T * k, H), sentinel))
    _assert_within(drows, ref, (u + (E32 if dtype == BF16 else 0.0)) * np.abs(ref) * (1 + u), "drows")
    assert np.array_equal(_np(drows)[~named.cpu().numpy()], ref[~named.cpu().numpy()])
    _assert_within(dw, dw_ref, (H + 1) * E32 * dw_size, "dw")


# (T, E, k): a softmax of one, of all, more slots than lanes, E not a multiple
# of anything, the largest E
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 384, 8), (7, 5, 5), (66, 333, 70), (129, 1024, 8), (3, 1024, 1024)])
def test_route_backward_matches_the_oracle(T, E, k):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"route backward T={T} E={E} k={k}")
    ids, w, _, _ = _routed(T, E, k, seed=2)
    dw = _rand((T, k), 5, FP32)
    out = torch.full((T, E), float("nan"), device="cuda")
    assert m.moe_route_backward(ids, w, dw, E, dlogits=out) is out
    i, w64, d64 = ids.cpu().numpy(), _np(w), _np(dw)
    ref = od.route_backward(i, w64, d64, E)
    # k products and additions in the sum, then a subtraction and a product
    size = w64 * (np.abs(d64) + np.sum(w64 * np.abs(d64), 1, keepdims=True))
    bound = np.zeros((T, E))
    np.put_along_axis(bound, i, (k + 4) * E32 * size, 1)
    _assert_within(out, ref, bound, "dlogits")


def test_ids_outside_the_experts_get_no_entry():
    from block_scaled_precision_amd import moe_mx as m
    ids = torch.tensor([[0, 9, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25, 0.25]], device="cuda")
    dw = torch.tensor([[1.0, 2.0, 4.0]], device="cuda")
    assert m.moe_route_backward(ids, w, dw, 4).tolist() == [[-0.5, 0.0, 0.0, 0.0]]  # 0.5 * (1 - 2)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("start,ld", [(0, 104), (8, 104), (1, 97), (3, 101)])
def test_strided_and_unaligned_rows(start, ld, dtype):
    """Views with a row stride, at and off 16-byte addresses, for every matrix;
    the memory between their rows stays as it was."""
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 19, 80, 8, 3
    print_flush(f"dispatch strided start={start} ld={ld} {dtype}")
    ids, w, off, order = _routed(T, E, k, seed=3)

    def view(rows, seed):
        buf = _rand((rows * ld + start + H,), seed, dtype)
        return buf, torch.as_strided(buf, (rows, H), (ld, 1), start)

    def check(buf, before, v, plain):
        assert torch.equal(v, plain)
        after = buf.clone()
        torch.as_strided(after, v.shape, v.stride(), start).copy_(torch.as_strided(before, v.shape, v.stride(), start))
        assert torch.equal(after, before)

    (_, x), (rbuf, rows) = view(T, 6), view(T * k, 7)
    before = rbuf.clone()
    _, row_of = m.moe_permute(x, order, off, k, rows=rows)
    check(rbuf, before, rows, m.moe_permute(x.contiguous(), order, off, k)[0])
    (_, g), (_, res), (ybuf, y) = view(T * k, 8), view(T, 9), view(T, 10)
    before = ybuf.clone()
    m.moe_unpermute(g, row_of, w, residual=res, y=y)
    check(ybuf, before, y, m.moe_unpermute(g.contiguous(), row_of, w, residual=res.contiguous()))
    before = ybuf.clone()
    m.moe_permute_backward(g, row_of, dx=y)
    check(ybuf, before, y, m.moe_permute_backward(g.contiguous(), row_of))
    (_, dy), (dbuf, drows) = view(T, 11), view(T * k, 12)
    before = dbuf.clone()
    _, dw = m.moe_unpermute_backward(dy, g, row_of, w, drows=drows)
    plain, dw2 = m.moe_unpermute_backward(dy.contiguous(), g.contiguous(), row_of, w)
    check(dbuf, before, drows, plain)
    # the element-wise and 16-byte forms add a dot product up in other orders
    size = (dy.double()[:, None] * g.double()[row_of.long()]).abs().sum(2)
    assert ((dw - dw2).abs() <= 2 * (H + 1) * E32 * size).all()


def test_capacity_drops_the_rows_past_it():
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 12, 32, 4, 2
    ids, w, off, order = _routed(T, E, k, seed=4)
    x = _rand((T, H), 13, BF16)
    full, row_of = m.moe_permute(x, order, off, k)
    for R in (T * k - 5, 0):
        rows, cut = m.moe_permute(x, order, off, k, rows=torch.empty((R, H), dtype=BF16, device="cuda"))
        assert torch.equal(rows, full[:R])
        assert torch.equal(cut, torch.where(row_of < R, row_of, torch.full_like(row_of, -1)))
        y = m.moe_unpermute(rows, cut, w)
        assert torch.equal(y, m.moe_unpermute(full[:R], row_of, w))  # rows past the matrix count as absent
        assert R > 0 or not y.any()
        drows, dw = m.moe_unpermute_backward(x, rows, cut, w)
        assert drows.shape == (R, H) and not dw[cut < 0].any()


def test_tokens_without_a_local_expert_and_empty_batches():
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 9, 48, 6, 2
    logits = gen.normal((T, E), 5, 30)
    logits[:, 3] = float("-inf")  # nobody chooses expert 3
    ids, w, off, order = m.moe_route(logits.cuda(), k)
    x = _rand((T, H), 14, FP32)
    rows, row_of = m.moe_permute(x, order, off, k, local_offset=3, local_count=1,
                                 rows=torch.full((T, H), 5.0, device="cuda"))
    assert (row_of == -1).all() and (rows == 5.0).all()
    assert not m.moe_permute_backward(rows, row_of).any()
    assert torch.equal(m.moe_unpermute(rows, row_of, w, residual=x), x)
    drows, dw = m.moe_unpermute_backward(x, rows, row_of, w, drows=torch.full((T, H), 6.0, device="cuda"))
    assert (drows == 6.0).all() and not dw.any()
    x0, none = x[:0], torch.empty((0, k), dtype=torch.int32, device="cuda")
    w0 = torch.empty((0, k), device="cuda")
    rows, row_of = m.moe_permute(x0, none.view(-1), torch.zeros_like(off), k)
    assert rows.shape == (0, H) and row_of.shape == (0, k)
    assert m.moe_unpermute(rows, row_of, w0).shape == (0, H)
    assert m.moe_route_backward(none, w0, w0, E).shape == (0, E)


def test_infinities_and_nan_of_named_rows_arrive():
    from block_scaled_precision_amd import moe_mx as m
    row_of = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.5], [1.0, 0.0]], device="cuda")
    for dtype in (BF16, FP32):
        rows = torch.ones((3, 16), dtype=dtype, device="cuda")
        rows[0, 3], rows[1, 5], rows[2, 7] = float("inf"), float("nan"), float("-inf")
        y = m.moe_unpermute(rows, row_of, w).float()
        assert y[0, 3] == float("inf") and torch.isnan(y[0, 5]) and y[1, 7] == float("-inf")
        assert torch.isfinite(y).sum() == 2 * 16 - 3


def test_gradients_against_differences():
    """Central differences of the forward operators.  unpermute is linear in
    rows and in w: a difference over a step of 1 is exact up to the roundings
    of the two fp32 outputs, (k + 2) e of each sum of magnitudes S <= H * k * 16
    * 16 / 16.  The router's weights have third derivatives below 1 in each
    logit, so their difference over h = 2^-5 is off by at most h^2 / 6 plus the
    weights' roundings (8 e each) over 2h, times the sum of |dw|."""
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 4, 24, 6, 3
    logits = (torch.arange(E).float().repeat(T, 1) * 0.25)[:, torch.randperm(E, generator=torch.Generator().manual_seed(1))].cuda()
    ids, w, off, order = m.moe_route(logits, k)
    x = _rand((T, H), 15, FP32)
    rows, row_of = m.moe_permute(x, order, off, k)
    dy = _rand((T, H), 16, FP32)
    drows, dw = m.moe_unpermute_backward(dy, rows, row_of, w)

    def loss(rows_, w_):
        return (m.moe_unpermute(rows_, row_of, w_).double() * dy.double()).sum().item()

    tol = 2 * (k + 2) * E32 * float((rows.abs().sum() + H) * dy.abs().max())
    for p, c in [(0, 0), (5, 11), (T * k - 1, H - 1)]:
        hi, lo_ = rows.clone(), rows.clone()
        hi[p, c] += 1.0
        lo_[p, c] -= 1.0
        step = (hi[p, c].double() - lo_[p, c].double()).item()
        assert abs((loss(hi, w) - loss(lo_, w)) / step - drows[p, c].item()) <= tol
    for t, j in [(0, 0), (2, 1), (3, 2)]:
        hi, lo_ = w.clone(), w.clone()
        hi[t, j] += 0.5
        lo_[t, j] -= 0.5
        step = (hi[t, j].double() - lo_[t, j].double()).item()
        assert abs((loss(rows, hi) - loss(rows, lo_)) / step - dw[t, j].item()) <= tol
    dx = m.moe_permute_backward(drows, row_of)
    for t, c in [(0, 0), (3, 7)]:
        def through(delta):
            xx = x.clone()
            xx[t, c] += delta
            return loss(m.moe_permute(xx, order, off, k)[0], w), xx[t, c].double().item()
        (a, xa), (b, xb) = through(1.0), through(-1.0)
        assert abs((a - b) / (xa - xb) - dx[t, c].item()) <= tol

    dlogits = m.moe_route_backward(ids, w, dw, E)
    h = 2.0 ** -5
    for t, e in [(0, int(ids[0, 0])), (1, int(ids[1, 2])), (3, int(ids[3, 1]))]:
        vals = []
        for s in (h, -h):
            lg = logits.clone()
            lg[t, e] += s
            i2, w2, _, _ = m.moe_route(lg, k)
            assert torch.equal(i2, ids)
            vals.append((w2.double() * dw.double()).sum().item())
        err = abs((vals[0] - vals[1]) / (2 * h) - dlogits[t, e].item())
        assert err <= (h * h / 6 + 8 * E32 / h + 8 * E32) * dw[t].abs().sum().item()


def _chain(m, x, logits, gain, dy, k, E):
    """Route, sort, scale each expert's rows, combine onto x; and all gradients."""
    ids, w, off, order = m.moe_route(logits, k)
    rows, row_of = m.moe_permute(x, order, off, k)
    h = rows * gain
    y = m.moe_unpermute(h, row_of, w, residual=x)
    dh, dw = m.moe_unpermute_backward(dy, h, row_of, w)
    dx = m.moe_permute_backward(dh * gain, row_of)
    return y, dx, m.moe_route_backward(ids, w, dw, E)


def test_chain_repeats_on_streams_and_in_a_replayed_graph():
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 70, 264, 12, 3
    print_flush("dispatch chain: streams and graph")
    sets = [tuple(_rand(s, 20 + i, FP32) for s in ((T, H), (T, E), (T * k, H), (T, H))) for i in range(3)]
    want = [_chain(m, x, lg, gain, dy, k, E) for x, lg, gain, dy in sets]
    torch.cuda.synchronize()
    again = _chain(m, *sets[0], k, E)
    assert all(torch.equal(a, b) for a, b in zip(again, want[0]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _chain(m, *sets[1], k, E)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(other, want[1]))
    bufs = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _chain(m, *bufs, k, E)
    for i in (1, 2, 0, 1):
        for b, t in zip(bufs, sets[i]):
            b.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        _chain(m, *sets[2], k, E)  # eager work between replays
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), f"replay of set {i}"


def test_prepared_calls_and_a_stream_argument():
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 40, 136, 10, 4
    ids, w, off, order = _routed(T, E, k, seed=6)
    x, dy = _rand((T, H), 40, BF16), _rand((T, H), 41, BF16)
    permute = m.OpCall(m.moe_permute, x, order, off, k)
    rows, row_of = permute()
    combine = m.OpCall(m.moe_unpermute, rows, row_of, w, residual=dy)
    y = combine()
    assert torch.equal(y, m.moe_unpermute(rows, row_of, w, residual=dy))
    x.mul_(2)  # the same buffers, new contents
    permute()
    assert combine() is y and torch.equal(y, m.moe_unpermute(rows, row_of, w, residual=dy))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = m.moe_unpermute(rows, row_of, w, residual=dy, stream=side)
    call = m.OpCall(m.moe_unpermute, rows, row_of, w, residual=dy, stream=side)
    y3 = call()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y2, y) and torch.equal(y3, y)


def test_overlapping_outputs_are_refused():
    from block_scaled_precision_amd import moe_mx as m
    T, H, E, k = 6, 32, 4, 2
    ids, w, off, order = _routed(T, E, k)
    x = _rand((T * k, H), 42, FP32)
    rows, row_of = m.moe_permute(x[:T], order, off, k)
    for call in (lambda: m.moe_permute(x[:T], order, off, k, rows=x),
                 lambda: m.moe_permute_backward(rows, row_of, dx=rows[:T]),
                 lambda: m.moe_unpermute(rows, row_of, w, residual=x[1:T + 1], y=x[:T]),
                 lambda: m.moe_unpermute_backward(x[:T], rows, row_of, w, drows=rows)):
        with pytest.raises(ValueError, match="overlaps"):
            call()


def test_sizes_past_32_bit_offsets():
    """Rows at element offsets beyond 2^32: the last rows of a matrix of 9.7 GB."""
    from block_scaled_precision_amd import moe_mx as m
    T, H, k, E = 3, 7168, 2, 4
    R = (1 << 32) // H + 80000
    print_flush(f"dispatch 64-bit offsets R={R}")
    rows = torch.empty((R, H), dtype=BF16, device="cuda")
    rows[-8:] = _rand((8, H), 43, BF16)
    row_of = torch.tensor([[R - 1, R - 8], [R - 3, -1], [R - 5, R]], dtype=torch.int32, device="cuda")
    w = torch.rand((T, k), device="cuda")
    dy = _rand((T, H), 44, BF16)
    small = torch.where((row_of >= 0) & (row_of < R), row_of - (R - 8), torch.full_like(row_of, -1))
    assert torch.equal(m.moe_unpermute(rows, row_of, w), m.moe_unpermute(rows[-8:], small, w))
    tail = rows[-8:].clone()
    want, want_dw = m.moe_unpermute_backward(dy, tail, small, w, drows=torch.zeros_like(tail))
    drows = torch.zeros((R, H), dtype=BF16, device="cuda")
    _, dw = m.moe_unpermute_backward(dy, rows, row_of, w, drows=drows)
    assert torch.equal(dw, want_dw) and torch.equal(drows[-8:], want)
