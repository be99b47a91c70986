"""moe_balance and moe_balance_backward on the GPU against the float64 oracle, whose last
results are the sums that bound fp32's error, in half steps (oracle/balance.py); counts and
tokens are exact.

Half steps do not count what falls below fp32's normal range, 2^-126.  In a gradient a p
(f - dot) + b lse p that is p (off by 2^-126 where the exponential or its quotient ends there),
the E terms of dot, and the few products that form the result: in all less than 2^-126 (E + 4)
(|a| + |b| (|lse| + 1) + 1), with |a| <= |dloss0| E, |b| <= 2 |dloss1|."""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from oracle import balance as ob
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

E32 = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _case(T, E, k, S, seed, std=1.0, masked=False):
    """logits, ids, mask, offsets; the ids of the largest logits, sequences of any length."""
    rng = np.random.default_rng(seed)
    logits = gen.normal((T, E), seed, 1, std=std)
    ids = torch.topk(logits, k, dim=1).indices.int()
    mask = torch.from_numpy(rng.random(T) < 0.7) if masked else None
    off = np.concatenate([[0], np.sort(rng.integers(0, T + 1, S - 1)), [T]])
    return logits, ids, mask, off


def _check(logits, ids, mask, off, S, *, whole=False, dloss=(0.7, -1.3), add=None, ld=None):
    from block_scaled_precision_amd import moe_mx as m
    T, E = logits.shape
    k = ids.shape[1]
    wide = torch.full((T, ld or E), float("nan"))
    wide[:, :E] = logits
    x = wide.cuda()[:, :E]
    so = None if whole else torch.from_numpy(np.asarray(off)).int().cuda()
    msk = None if mask is None else mask.cuda()
    loss, counts, tokens, lse = m.moe_balance(x, ids.cuda(), mask=msk, seq_offsets=so)
    ref = ob.balance(_np(logits), ids.numpy(), S, off, None if mask is None else mask.numpy())
    assert np.array_equal(counts.cpu().numpy(), ref[1]) and np.array_equal(tokens.cpu().numpy(), ref[2])
    got, want, size = _np(lse), ref[3], ref[5]
    live = want > -np.inf
    assert np.array_equal(got == -np.inf, ~live)
    assert (np.abs(got - want)[live] <= size[live] * E32).all()
    assert (np.abs(_np(loss) - ref[0]) <= ref[4] * E32).all(), (_np(loss), ref[0], ref[4] * E32)
    d = torch.tensor(dloss, dtype=F32)
    g = m.moe_balance_backward(d.cuda(), x, counts, tokens, lse, k, seq_offsets=so,
                               add=None if add is None else add.cuda())
    gref, gsize = ob.balance_backward(_np(d), _np(logits), ref[1], ref[2], k, off, None if mask is None else mask.numpy(),
                                      None if add is None else _np(add))
    top = np.abs(want[live]).max(initial=0.0) + 1
    tiny = 2.0 ** -126 * (E + 4) * (abs(dloss[0]) * E + 2 * abs(dloss[1]) * top + 1)
    bad = ~(np.abs(_np(g) - gref) <= gsize * E32 + tiny)
    assert not bad.any(), (np.argwhere(bad)[:3], _np(g)[bad][:3], gref[bad][:3], (gsize * E32)[bad][:3])
    return loss, counts, tokens, lse, g


SIZES = [(1, 1, 1, 1), (1, 8, 2, 1), (3, 1, 1, 2), (5, 7, 3, 1), (64, 64, 8, 1), (128, 256, 8, 4), (129, 256, 8, 4), (128, 33, 5, 5),
         (200, 1024, 8, 3), (333, 384, 6, 1), (1000, 128, 4, 7), (1000, 65, 2, 300), (2049, 16, 1, 2), (700, 513, 16, 9),
         (4096, 8, 8, 1), (90, 1000, 1000, 2)]


@pytest.mark.parametrize("T,E,k,S", SIZES)
def test_losses_counts_and_gradients(T, E, k, S):
    print_flush(f"moe_balance T={T} E={E} k={k} S={S}")
    for masked in (False, True):
        logits, ids, mask, off = _case(T, E, k, S, T + E + S, masked=masked)
        _check(logits, ids, mask, off, S)
        add = gen.normal((T, E), T, 3)
        _check(logits, ids, mask, off, S, add=add, ld=E + 3)
        _check(logits, ids, mask, off, S, add=add, ld=(E + 7) // 4 * 4)
    if S == 1:
        _check(logits, ids, None, off, 1, whole=True)
    # of any size: one probability is 1, the others underflow
    logits, ids, mask, off = _case(T, E, k, S, 5, std=40.0)
    _check(logits, ids, mask, off, S)


def _draw(n, seed=20261210):
    rng = np.random.default_rng(seed)
    out = []
    for i in range(n):
        E = int(np.exp(rng.uniform(0, np.log(1025))))
        T = int(np.exp(rng.uniform(0, np.log(3000))))
        out.append((T, E, int(rng.integers(1, min(E, 12) + 1)), int(np.exp(rng.uniform(0, np.log(40)))), i))
    return out


@pytest.mark.parametrize("T,E,k,S,i", _draw(30))
def test_drawn_sizes(T, E, k, S, i):
    print_flush(f"moe_balance drawn T={T} E={E} k={k} S={S}")
    logits, ids, mask, off = _case(T, E, k, S, i, std=3.0, masked=i % 2 == 0)
    _check(logits, ids, mask, off, S, add=gen.normal((T, E), i, 3) if i % 3 == 0 else None, ld=E + i % 5)


@pytest.mark.parametrize("T", [100, 600])
def test_tokens_that_do_not_count(T):
    """Padding of any content, tokens before the first and behind the last sequence, empty
    sequences, rows of -inf, single -inf logits, ids out of range, offsets past the ends."""
    E, k = 96, 4
    logits, ids, _, _ = _case(T, E, k, 1, 3)
    mask = torch.ones(T, dtype=torch.bool)
    mask[5:40] = False
    logits[5], logits[6], logits[7, 3] = float("nan"), INF, -INF
    logits[50] = -INF
    logits[51, ::2] = -INF
    logits[60, 1:] = -INF
    logits[61, 1:] = torch.finfo(F32).min
    logits[62, 5] = torch.finfo(F32).min
    logits[0], logits[T - 1] = float("nan"), float("nan")
    ids[70] = torch.tensor([-1, E, 2 ** 31 - 1, -2 ** 31])
    ids[71] = ids[71, 0].item()  # one expert four times
    off = [2, 2, 30, 45, 45, 80, T - 3, T - 3]
    _, _, _, lse, g = _check(logits, ids, mask, off, 7)
    assert (g[5:40] == 0).all() and (g[:2] == 0).all() and (g[50] == 0).all()
    _check(logits[2:T - 1], ids[2:T - 1], mask[2:T - 1], [-5, 2, 30, T + 99], 3)
    nothing = torch.zeros(T, dtype=torch.bool)
    loss, counts, tokens, lse, g = _check(logits, ids, nothing, off, 7)
    assert (loss == 0).all() and not counts.any() and not tokens.any() and (lse == -INF).all() and (g == 0).all()


@pytest.mark.parametrize("T", [20, 500])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_a_counted_token_without_a_distribution(T, bad):
    """Both losses become NaN, counts and the other tokens' lse stay."""
    from block_scaled_precision_amd import moe_mx as m
    logits, ids, _, off = _case(T, 32, 2, 2, 9)
    want = m.moe_balance(logits.cuda(), ids.cuda(), seq_offsets=torch.tensor(off).int().cuda())
    logits[T // 2, 3] = bad
    loss, counts, tokens, lse = m.moe_balance(logits.cuda(), ids.cuda(), seq_offsets=torch.tensor(off).int().cuda())
    assert torch.isnan(loss).all() and torch.equal(counts, want[1]) and torch.equal(tokens, want[2])
    keep = torch.arange(T) != T // 2
    assert torch.equal(lse.cpu()[keep], want[3].cpu()[keep])


@pytest.mark.parametrize("off", [[0, 400, 100, 300], [7, 3, 2, 1], [-2 ** 31, 2 ** 31 - 1, 0, 5], [300, 300, 0, 300]])
def test_offsets_out_of_order_stay_in_bounds(off):
    """Outputs lie between guard areas; each call ends."""
    from block_scaled_precision_amd import moe_mx as m
    for T, S in ((300, 3), (90, 3)):
        logits, ids, _, _ = _case(T, 40, 3, 1, 4)
        buf = torch.full((3 * S, 40), -9, dtype=torch.int32, device="cuda")
        lse = torch.full((3 * T,), 9.0, device="cuda")
        tok = torch.full((3, S + 2), -9, dtype=torch.int32, device="cuda")
        out = torch.full((3 * T, 40), 9.0, device="cuda")
        so = torch.tensor(off, dtype=torch.int32).cuda()
        m.moe_balance(logits.cuda(), ids.cuda(), seq_offsets=so, counts=buf[S:2 * S], tokens=tok[1], lse=lse[T:2 * T])
        m.moe_balance_backward(torch.ones(2).cuda(), logits.cuda(), buf[S:2 * S], tok[1], lse[T:2 * T], 3, seq_offsets=so,
                               dlogits=out[T:2 * T])
        torch.cuda.synchronize()
        for t, n in ((buf, S), (lse, T), (tok, 1), (out, T)):
            guard = -9 if t.dtype == torch.int32 else 9.0
            assert (t[:n] == guard).all() and (t[2 * n:] == guard).all()


@pytest.mark.parametrize("T,E,k,S", [(60, 64, 4, 2), (400, 64, 4, 3)])
def test_gradient_against_differences(T, E, k, S):
    """Central differences of the oracle's float64 losses, along directions with entries up to
    1: their error is h^2 / 6 times the third derivative, which is at most 8 times the first
    loss (here below 3) and 2 (6 lse + 3 * 2) for the second (lse below 7), and the fp32 error
    of the gradient."""
    logits, ids, mask, off = _case(T, E, k, S, 8, masked=True)
    d = (0.7, -1.3)
    g = _np(_check(logits, ids, mask, off, S, dloss=d)[-1])
    _, gsize = ob.balance_backward(np.float32(d).astype(float), _np(logits), *ob.balance(_np(logits), ids.numpy(), S, off,
                                                                                       mask.numpy())[1:3], k, off,
                                   mask.numpy())
    rng = np.random.default_rng(1)
    h = 1e-4
    for _ in range(8):
        v = rng.standard_normal((T, E))
        v /= np.abs(v).max()

        def at(step):
            loss = ob.balance(_np(logits) + step * v, ids.numpy(), S, off, mask.numpy())[0]
            return np.float32(d[0]) * loss[0] + np.float32(d[1]) * loss[1]
        diff = (at(h) - at(-h)) / (2 * h)
        assert abs(diff - np.sum(g * v)) <= E32 * np.sum(gsize * np.abs(v)) + 100 * h * h + 1e-12 / h


def test_add_in_place_strides_and_broadcast_gradients():
    from block_scaled_precision_amd import moe_mx as m
    T, E, k = 300, 72, 4
    logits, ids, _, _ = _case(T, E, k, 1, 6)
    x = logits.cuda()
    out = m.moe_balance(x, ids.cuda())
    add = gen.normal((T, E), 7, 3).cuda()
    want = m.moe_balance_backward(torch.ones(2).cuda(), x, *out[1:], k, add=add)
    buf = add.clone()
    assert m.moe_balance_backward(torch.ones(2).cuda(), x, *out[1:], k, add=buf, dlogits=buf) is buf
    assert torch.equal(buf, want)
    wide = torch.full((T, E + 8), 5.0, device="cuda")
    wide[:, 3:E + 3] = add
    m.moe_balance_backward(torch.ones(2).cuda(), x, *out[1:], k, add=wide[:, 3:E + 3], dlogits=wide[:, 3:E + 3])
    # another alignment may sum in another order
    ref, size = ob.balance_backward([1.0, 1.0], _np(logits), out[1].cpu().numpy(), out[2].cpu().numpy(), k, [0, T],
                                    add=_np(add))
    for got in (want, wide[:, 3:E + 3]):
        assert (np.abs(_np(got) - ref) <= size * E32).all()
    assert (wide[:, :3] == 5).all() and (wide[:, E + 3:] == 5).all()


def test_no_tokens():
    from block_scaled_precision_amd import moe_mx as m
    x, ids = torch.zeros((0, 16), device="cuda"), torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, tokens, lse = m.moe_balance(x, ids, seq_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert (loss == 0).all() and counts.shape == (3, 16) and not counts.any() and not tokens.any() and lse.shape == (0,)
    assert m.moe_balance_backward(loss, x, counts, tokens, lse, 2,
                                  seq_offsets=torch.zeros(4, dtype=torch.int32, device="cuda")).shape == (0, 16)


def test_results_repeat_and_calls_at_once_and_captured():
    """Prepared calls on two streams at the same time, then captured ones replayed among eager
    work: bit for bit the same."""
    from block_scaled_precision_amd import moe_mx as m
    for T, E, k, S in ((100, 256, 8, 2), (5000, 256, 8, 6), (30000, 64, 6, 1)):
        print_flush(f"moe_balance at once T={T}")
        data = []
        for i in range(2):
            logits, ids, _, off = _case(T, E, k, S, 20 + i)
            data.append((logits.cuda(), ids.cuda(), torch.tensor(off).int().cuda()))
        want = [m.moe_balance(x, ids, seq_offsets=o) for x, ids, o in data]
        calls = [m.OpCall(m.moe_balance, x, ids, seq_offsets=o) for x, ids, o in data]
        streams = [torch.cuda.Stream() for _ in data]
        torch.cuda.synchronize()
        for _ in range(20):
            for call, st in zip(calls, streams):
                with torch.cuda.stream(st):
                    call()
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            assert all(torch.equal(g, r) for g, r in zip(call(), w))
        graphs = []
        for call, (x, _, o) in zip(calls, data):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = call()
                grad = m.moe_balance_backward(torch.ones(2, device="cuda"), x, *out[1:], k, seq_offsets=o)
            graphs.append((g, out, grad))
        for i in (0, 1, 1, 0, 1):
            g, out, grad = graphs[i]
            for t in (*out, grad):
                t.zero_()
            g.replay()
            other = m.moe_balance(data[1 - i][0], data[1 - i][1], seq_offsets=data[1 - i][2])
            eager = m.moe_balance_backward(torch.ones(2, device="cuda"), data[i][0], *want[i][1:], k,
                                           seq_offsets=data[i][2])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i])) and torch.equal(grad, eager)
            assert all(torch.equal(a, b) for a, b in zip(other, want[1 - i]))


def test_more_chunks_than_a_short_batch_has():
    """Rows past 512 chunks of 256: the sums in fp32 stay as short as the oracle's bound takes
    them to be."""
    T, E, k, S = 150001, 5, 2, 3
    print_flush(f"moe_balance T={T}")
    logits, ids, mask, off = _case(T, E, k, S, 31, masked=True)
    _check(logits, ids, mask, off, S)


def test_most_sequences():
    """2^20 sequences of 3 tokens, more than are held in LDS, each with an expert of its own."""
    from block_scaled_precision_amd import moe_mx as m
    S, E = 1 << 20, 4
    T = 3 * S
    s = torch.arange(T, device="cuda") // 3
    x = torch.zeros((T, E), device="cuda")
    ids = (s % E).int()[:, None].contiguous()
    so = 3 * torch.arange(S + 1, device="cuda", dtype=torch.int32)
    loss, counts, tokens, lse = m.moe_balance(x, ids, seq_offsets=so)
    want = 3 * torch.nn.functional.one_hot(torch.arange(S, device="cuda") % E, E).int()
    assert torch.equal(counts, want) and (tokens[:S] == 3).all() and tokens[S:].tolist() == [T, S]
    # every p is 1/4, the loss 1; half steps as the oracle counts them, with |x - max| = 0
    top = np.log(4.0)
    lse_steps = 28 + 2 * top + 2 * top
    assert abs(loss[0].item() - 1) <= (28 + 80 + 2) * E32 and (lse - top).abs().max().item() <= lse_steps * E32
    assert abs(loss[1].item() - top ** 2) <= (2 * top * lse_steps + 66 * top ** 2) * E32
    g = m.moe_balance_backward(torch.tensor([1.0, 0.0]).cuda(), x, counts, tokens, lse, 1, seq_offsets=so)
    # E / (S 3) p_e (f_e - 1/4): f is 1 for one expert
    ref = E / T * 0.25 * ((want[s] > 0).double() - 0.25)
    steps = top + lse_steps + 8
    assert ((g.double() - ref).abs() <= E / T * 0.25 * ((steps + 8) * 1.25 + 0.25 * (steps + 24)) * E32
            + 2 * ref.abs() * E32).all()


def test_rows_past_32_bit_offsets():
    """Logits of more than 2^32 bytes: the last tokens of a long batch (one sequence of their
    own) against the same tokens alone."""
    from block_scaled_precision_amd import moe_mx as m
    E, k, n = 1024, 2, 100
    T = (1 << 21) + n
    x = torch.zeros((T, E), device="cuda")
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    logits, few, _, _ = _case(n, E, k, 1, 30)
    x[-n:], ids[-n:] = logits.cuda(), few.cuda()
    so = torch.tensor([0, T - n, T]).int().cuda()
    _, counts, tokens, lse = m.moe_balance(x, ids, seq_offsets=so)
    alone = m.moe_balance(x[-n:], ids[-n:])
    assert torch.equal(counts[1], alone[1][0]) and tokens.tolist() == [T - n, n, T, 2]
    assert counts[0, 0].item() == (T - n) * k and torch.equal(lse[-n:], alone[3])
    g = m.moe_balance_backward(torch.tensor([2.0, 0.0]).cuda(), x, counts, tokens, lse, k, seq_offsets=so)
    one = m.moe_balance_backward(torch.tensor([1.0, 0.0]).cuda(), x[-n:], *alone[1:], k)
    # 2 / 2 sequences: the same factors
    assert torch.equal(g[-n:], one)


def test_a_training_step_of_an_expert_layer():
    """Router, losses, permutation, experts in MXFP4, combination; backward through the
    experts' operands and through the router, whose two gradients meet in one call.  Every
    step against float64 on the step's own inputs, so that no choice of experts or codes has
    to agree across steps."""
    from block_scaled_precision_amd import moe_mx as m
    T, H, I, E, k = 200, 256, 128, 16, 4
    x = gen.normal((T, H), 70, 1).to(BF16).cuda()
    wr = gen.normal((E, H), 70, 2, std=0.1).to(BF16)
    logits = (x.float() @ wr.float().cuda().T).contiguous()
    w13 = m.mx4_quantize(gen.normal((E, 2 * I, H), 70, 3, std=0.1).to(BF16).cuda())
    w2src = gen.normal((E, H, I), 70, 4, std=0.1).to(BF16).cuda()
    w2 = m.mx4_quantize(w2src)
    so = torch.tensor([0, 120, 120, T]).int().cuda()

    def val(t):
        return _np(m.mx4_dequantize(*t, dtype=F32))

    def near(got, a, b):  # one rounding to bf16 and the fp32 sum of a row
        ref, size = a @ b.T, np.abs(a) @ np.abs(b).T
        assert (np.abs(_np(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * 2 * a.shape[1] * E32 * size).all()

    ids, weights, offsets, assign = m.moe_route(logits, k)
    loss, counts, tokens, lse = m.moe_balance(logits, ids, seq_offsets=so)
    assert torch.equal(counts.sum(0), offsets.diff())
    rows, row_of = m.moe_permute(x, assign, offsets, k)
    xq = m.mx4_quantize(rows)
    off = offsets.cpu().numpy()
    up = m.mx4_linear(xq[0], w13[0][:, I:], w13[1][:, I:], a_scale=xq[1], expert_offsets=offsets)
    act = m.mx4_linear(xq[0], w13[0][:, :I], w13[1][:, :I], a_scale=xq[1], expert_offsets=offsets, fn="silu", mul=up)
    aq = m.mx4_quantize(act)
    y = m.mx4_linear(aq[0], w2[0], w2[1], a_scale=aq[1], expert_offsets=offsets)
    xv, av, w13v, w2v = val(xq), val(aq), val(w13), val(w2)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        near(up[s], xv[s], w13v[e, I:])
        near(y[s], av[s], w2v[e])
    out = m.moe_unpermute(y, row_of, weights)
    terms = _np(weights)[:, :, None] * _np(y)[row_of.cpu().numpy()]
    ref, size = terms.sum(1), np.abs(terms).sum(1)
    assert (np.abs(_np(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2 * (k + 1) * E32 * size).all()
    # backward: the rows' gradients, through the transposed weights, and per expert dW
    dy, dw = m.moe_unpermute_backward(gen.normal((T, H), 70, 6).to(BF16).cuda(), y, row_of, weights)
    dq, wt = m.mx4_quantize(dy), m.mx4_quantize(w2src, transpose=True)
    da = m.mx4_linear(dq[0], wt[0], wt[1], a_scale=dq[1], expert_offsets=offsets)
    dv, wtv = val(dq), val(wt)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        near(da[s], dv[s], wtv[e])
        if off[e] < off[e + 1]:
            p, q = m.mx4_quantize(dy[s], transpose=True), m.mx4_quantize(act[s], transpose=True)
            near(m.mx4_linear(p[0], q[0], q[1], a_scale=p[1]), val(p), val(q))
    # the router: the losses' gradient on top of the weights'
    through = m.moe_route_backward(ids, weights, dw, E)
    d = torch.tensor([0.01, 0.001], device="cuda")
    got = m.moe_balance_backward(d, logits, counts, tokens, lse, k, seq_offsets=so, add=through)
    ref, size = ob.balance_backward(_np(d), _np(logits), counts.cpu().numpy(), tokens.cpu().numpy(), k, so.tolist(),
                                    add=_np(through))
    assert (np.abs(_np(got) - ref) <= size * E32).all()
