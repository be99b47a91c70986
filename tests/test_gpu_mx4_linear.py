"""mx4_linear on the GPU against the float64 oracle.

Exact cases: E2M1 codes with scale code 127 on both sides, integer biases and
residuals, products and partial sums multiples of 1/4 below 2^24 / 4: v + residual is
exact and its one rounding has to agree bit for bit with the oracle's.  bf16 rows of
integers are quantized by both sides first, which is exact arithmetic too.

Bounded cases: as for mx_linear, with e = 2^-24 for every fp32 operation and u = 2^-8
for the rounding to bf16 (tests/test_gpu_linear.py derives it); the 64 products of an
MFMA are exact in fp32's range (4 + 4 bits), so the sum's error is an accumulation's.
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from oracle import gemm as og
from oracle import mx, mx4
from tests.conftest import has_gpu
from tests.helpers import print_flush
from tests.test_gpu_linear import BF16, _bound, _ints, _np, _same_bits

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]


def _codes(shape, K, seed, scales=None):
    c = gen.random_bytes((*shape, K // 2), seed, 91)
    if scales is None:
        return c, torch.full((*shape, K // 32), 127, dtype=torch.uint8)
    g = torch.Generator().manual_seed(seed)
    return c, torch.randint(*scales, (*shape, K // 32), generator=g, dtype=torch.uint8)


def _offsets(M, G, seed):
    rng = np.random.default_rng(seed)
    return np.concatenate([[0], np.sort(rng.integers(0, M + 1, G - 1)), [M]]) if G else None


# (kernel, rows of its tiles, M, N, K, groups): every kernel that a call can take, dense and
# grouped, K a multiple of 256 and not, more items than workgroups and a part of one, N off the
# column blocks; tests/test_mx4_plan.py holds them against the choice
CASES = [
    ("few", 16, 1, 8, 128, 0), ("few", 16, 1, 4096, 7168, 0), ("few", 16, 5, 264, 384, 0), ("few", 16, 16, 1032, 1152, 0),
    ("few", 16, 8, 520, 4736, 0), ("few", 16, 8, 136, 10240, 0), ("few", 16, 2, 72, 16384, 0), ("few", 16, 16, 264, 2048, 6),
    ("few", 16, 33, 520, 640, 6), ("few", 16, 3, 72, 128, 2), ("few", 16, 20, 136, 896, 40), ("few", 16, 100, 40, 256, 1),
    ("tile", 64, 300, 2056, 512, 0), ("tile", 64, 700, 1032, 1152, 0), ("tile", 64, 4200, 2056, 640, 0),
    ("tile", 64, 700, 4104, 1152, 1), ("tile", 64, 4200, 1032, 512, 40), ("tile", 64, 1500, 1032, 2048, 6),
    ("tile", 64, 300, 4104, 512, 40),
    ("tile", 128, 1500, 4104, 512, 0), ("tile", 128, 9000, 1288, 640, 0), ("tile", 128, 9000, 1288, 896, 0),
    ("tile", 128, 4200, 1544, 640, 0), ("tile", 128, 9000, 4104, 640, 0), ("tile", 128, 3000, 2056, 512, 6),
    ("tile", 128, 9000, 264, 1152, 40), ("tile", 128, 4200, 1032, 640, 1), ("tile", 128, 9300, 4104, 512, 3),
    ("tile", 256, 3000, 4104, 1920, 0), ("tile", 256, 6000, 2056, 2176, 0), ("tile", 256, 9300, 2568, 3200, 0),
    ("tile", 256, 1900, 4104, 1920, 1), ("tile", 256, 6000, 4104, 1664, 3),
    ("ranges", 64, 64, 1032, 7168, 0), ("ranges", 64, 300, 2056, 7168, 0), ("ranges", 64, 100, 4104, 7040, 0),
    ("ranges", 64, 500, 520, 7168, 0),
    ("widen", 0, 700, 1032, 128, 0), ("widen", 0, 1500, 520, 384, 0),
    ("widen", 0, 3000, 1032, 128, 6),
]
IDS = [f"{k}{r}_{M}x{N}x{K}_g{G}" for k, r, M, N, K, G in CASES]


@pytest.mark.parametrize("kernel,rows,M,N,K,G", CASES, ids=IDS)
def test_exact_products_are_bit_identical(kernel, rows, M, N, K, G):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear exact {kernel}{rows} M={M} N={N} K={K} G={G}")
    (a, asc), (w, wsc) = _codes((M,), K, 0), _codes((G, N) if G else (N,), K, 1)
    ab = _ints((M, K), 0, 20)
    bias, res = _ints((G, N) if G else (N,), 1, 22, torch.float32), _ints((M, N), 2, 23)
    mul = 2.0 ** gen.small_integers((M, N), 3, 24, -2, 2).float()
    off = _offsets(M, G, M + N)
    kw = dict(expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    w_, s_, wn, sn = w.cuda(), wsc.cuda(), w.numpy(), wsc.numpy()
    ref, _, _ = mx4.mx4_linear(a.numpy(), wn, sn, a_scale=asc.numpy(), offsets=off, residual=_np(res))
    _same_bits(m.mx4_linear(a.cuda(), w_, s_, a_scale=asc.cuda(), residual=res.cuda(), **kw), ref, "codes, residual")
    ref, _, _ = mx4.mx4_linear(_np(ab), wn, sn, offsets=off)
    _same_bits(m.mx4_linear(ab.cuda(), w_, s_, **kw), ref, "bf16 rows")
    ref, _, _ = mx4.mx4_linear(a.numpy(), wn, sn, a_scale=asc.numpy(), offsets=off, bias=_np(bias.to(BF16)), mul=_np(mul))
    out = mul.to(BF16).cuda()
    assert m.mx4_linear(a.cuda(), w_, s_, a_scale=asc.cuda(), bias=bias.to(BF16).cuda(), mul=out, out=out, **kw) is out
    _same_bits(out, ref, "bias, mul in place")
    ref, _, _ = mx4.mx4_linear(a.numpy(), wn, sn, a_scale=asc.numpy(), offsets=off, bias=_np(bias), fn="relu2")
    _same_bits(m.mx4_linear(a.cuda(), w_, s_, a_scale=asc.cuda(), bias=bias.cuda(), fn="relu2", **kw),
               np.where(np.abs(ref) < 2.0 ** 20, ref, np.nan), "bias, relu2")


SOME = [c for c in CASES if c[2] * c[3] <= 1 << 21]


@pytest.mark.parametrize("fn", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("kernel,rows,M,N,K,G", SOME, ids=[i for i, c in zip(IDS, CASES) if c in SOME])
def test_activations_within_their_bound(kernel, rows, M, N, K, G, fn):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear {fn} {kernel}{rows} M={M} N={N} K={K} G={G}")
    a = gen.normal((M, K), 4, 25).to(BF16)
    w, s = _codes((G, N) if G else (N,), K, 4, scales=(118, 123))
    bias = gen.normal((G, N) if G else (N,), 4, 26)
    mul, res = gen.normal((M, N), 4, 27).to(BF16), gen.normal((M, N), 4, 28).to(BF16)
    off = _offsets(M, G, M + N)
    offd = None if off is None else torch.from_numpy(off).int().cuda()
    rows_bias = _np(bias) * np.ones((M, 1)) if off is None else np.repeat(_np(bias), np.diff(off), axis=0)
    for mu, re in ((None, None), (mul, None), (None, res), (mul, res)):
        got = m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), bias=bias.cuda(), fn=fn, expert_offsets=offd,
                           mul=None if mu is None else mu.cuda(), residual=None if re is None else re.cuda())
        mu64 = np.ones((M, N)) if mu is None else _np(mu)
        re64 = np.zeros((M, N)) if re is None else _np(re)
        ref, size, v = mx4.mx4_linear(_np(a), w.numpy(), s.numpy(), bias=_np(bias), fn=fn, mul=mu64, residual=re64,
                                      offsets=off)
        d = np.abs(_np(got) - ref)
        bound = _bound(fn, K, v, size, rows_bias, mu64, re64, ref)
        assert (d <= bound).all(), f"{(d > bound).sum()} out of bounds, worst ratio {(d / bound).max():.2f}"


PICKED = [(5, 264, 128), (1900, 136, 128), (20, 520, 384), (300, 2056, 640), (700, 1032, 1152), (3, 64, 3200),
          (2100, 2056, 896), (3000, 4104, 640), (400, 4104, 3584)]


@pytest.mark.parametrize("G", [0, 5])
@pytest.mark.parametrize("M,N,K", PICKED)
def test_every_code_meets_its_scales(M, N, K, G):
    """Row m holds one nonzero code, at k = 33 m mod K, in a block of scale 2^(m mod 9 - 4), so
    out[m, n] is a weight times its block's scale (of any size) and that value."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear picked M={M} N={N} K={K} G={G}")
    w, s = _codes((G, N) if G else (N,), K, 18, scales=(60, 190))
    rows, k = torch.arange(M), 33 * torch.arange(M) % K
    a = torch.zeros((M, K // 2), dtype=torch.uint8)
    a[rows, k // 2] = (2 << 4 * (k % 2)).to(torch.uint8)  # 1.0
    asc = torch.randint(100, 150, (M, K // 32), generator=torch.Generator().manual_seed(5), dtype=torch.uint8)
    asc[rows, k // 32] = (123 + rows % 9).to(torch.uint8)
    off = torch.tensor([0, 0, M // 3, M // 3 + 1, M - M // 4, M]).int() if G else None
    got = _np(m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), a_scale=asc.cuda(),
                           expert_offsets=None if off is None else off.cuda()))
    for g, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist()) if G else [(0, M)]):
        if lo == hi:
            continue
        weights = mx4.values((w[g] if G else w).numpy(), (s[g] if G else s).numpy())
        ref = weights[:, k[lo:hi].numpy()].T * 2.0 ** (rows[lo:hi].numpy() % 9 - 4)[:, None]
        assert np.array_equal(got[lo:hi], ref), f"group {g}"


@pytest.mark.parametrize("counts", [[0, 1, 15, 0, 16, 17, 33, 0], [64, 65, 128, 129, 0, 255, 256, 257, 10], [37], [0, 0, 0, 50],
                                    [50, 0, 0], [0, 0], [700, 3, 900]], ids=str)
@pytest.mark.parametrize("N,K", [(512, 1024), (264, 640), (72, 384), (2056, 512)])
def test_groups_are_bit_identical(N, K, counts):
    """Rows sorted by group; offsets that do not start at 0, rows behind the last group (NaN
    in A) left as they were, weights at a stride (the gate half of [gate; up])."""
    from block_scaled_precision_amd import moe_mx as m
    G, P, tail = len(counts), sum(counts), 5
    M = P + tail
    print_flush(f"mx4_linear groups {counts} N={N} K={K}")
    offsets = np.concatenate([[0], np.cumsum(counts)]) + 11
    a, (w, s) = _ints((M, K), 5, 20), _codes((G, 2 * N), K, 5)
    bias, res = _ints((G, N), 6, 22, torch.float32), _ints((M, N), 7, 23)
    ref, _, _ = mx4.mx4_linear(_np(a), w.numpy()[:, :N], s.numpy()[:, :N], bias=_np(bias), residual=_np(res),
                               offsets=offsets)
    a[P:] = float("nan")
    off = torch.from_numpy(offsets).int().cuda()
    for given in (False, True):
        out = torch.full((M, N), 33.0, dtype=BF16, device="cuda")
        x, sc = m.mx4_quantize(a.cuda()) if given else (a.cuda(), None)
        m.mx4_linear(x, w.cuda()[:, :N], s.cuda()[:, :N], a_scale=sc, bias=bias.cuda(), residual=res.cuda(),
                     expert_offsets=off, out=out)
        torch.cuda.synchronize()
        assert (out[P:] == 33.0).all()
        _same_bits(out, ref, f"given {given}")


@pytest.mark.parametrize("M,N,K", [(40, 64, 256), (300, 520, 640), (3000, 2056, 512)])
def test_offsets_out_of_order_or_range_stay_in_bounds(M, N, K):
    """Whatever the offsets hold, nothing outside [M, N] is written: out lies between two
    guard areas."""
    from block_scaled_precision_amd import moe_mx as m
    a, (w, s) = _ints((M, K), 8, 20), _codes((4, N), K, 8)
    buf = torch.full((3 * M, N), 9.0, dtype=BF16, device="cuda")
    for off in ([0, 1000, 5, 60, 80], [7, 3, 2, 1, 0], [-2 ** 31, 2 ** 31 - 1, 0, 5, 9], [0, 10, 10, 2, 30]):
        m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), expert_offsets=torch.tensor(off, dtype=torch.int32).cuda(),
                     out=buf[M:2 * M])
        torch.cuda.synchronize()
        assert (buf[:M] == 9.0).all() and (buf[2 * M:] == 9.0).all()


@pytest.mark.parametrize("M,N,K", [(3, 64, 256), (70, 264, 640), (700, 1032, 640), (3000, 4104, 512)])
def test_nan_scales_and_infinite_results(M, N, K):
    """A NaN scale makes its row or column NaN and no other; sums past bf16's range are
    infinite."""
    from block_scaled_precision_amd import moe_mx as m
    (a, asc), (w, s) = _codes((M,), K, 30), _codes((N,), K, 31)
    a[:], w[:] = a & 0x77 | 0x22, w & 0x77 | 0x22  # all above zero
    asc[M // 2, K // 64], s[N // 3, 0] = 255, 255
    asc[0], s[1] = 200, 240  # row 0 times column 1: 2^(73 + 113) and more
    got = _np(m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), a_scale=asc.cuda()))
    bad = np.zeros((M, N), dtype=bool)
    bad[M // 2], bad[:, N // 3] = True, True
    assert np.isnan(got[bad]).all() and not np.isnan(got[~bad]).any()
    if M > 2:
        assert np.isinf(got[0, 1])


@pytest.mark.parametrize("M,N,K,G", [(3, 72, 256, 0), (300, 2056, 640, 0), (1500, 4104, 512, 0), (3000, 4104, 512, 0), (3000, 520, 640, 40),
                                     (3000, 2056, 512, 6), (300, 4104, 512, 40)])
def test_biases_of_any_alignment(M, N, K, G):
    """Either type, from every address of the type; the bias differs in every column and group,
    and NaN stands before and behind it."""
    from block_scaled_precision_amd import moe_mx as m
    w, s = (t.cuda() for t in _codes((G, N) if G else (N,), K, 50))
    a, asc = _codes((M,), K, 51)
    off = _offsets(M, G, M)
    kw = dict(a_scale=asc.cuda(), expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    n = max(G, 1) * N
    values = ((torch.arange(n) * 37) % 509 - 254).float()
    for dtype, step in ((torch.float32, 4), (BF16, 2)):
        ref, _, _ = mx4.mx4_linear(a.numpy(), w.cpu().numpy(), s.cpu().numpy(), a_scale=asc.numpy(), offsets=off,
                                   bias=values.to(dtype).double().numpy().reshape((G, N) if G else (N,)))
        for at in range(0, 16, step):
            buf = torch.full((n + 16,), float("nan"), dtype=dtype, device="cuda")
            view = buf[at // step:at // step + n]
            view.copy_(values)
            _same_bits(m.mx4_linear(a.cuda(), w, s, bias=view.view((G, N) if G else (N,)), **kw), ref, f"{dtype} at {at}")


def test_no_rows_and_aliases():
    from block_scaled_precision_amd import moe_mx as m
    a, (w, s) = _ints((0, 256), 9, 20), _codes((64,), 256, 9)
    assert m.mx4_linear(a.cuda(), w.cuda(), s.cuda()).shape == (0, 64)
    for M, N, K in ((20, 64, 256), (1500, 1032, 512)):
        (w, s) = _codes((N,), K, 9)
        a, res = _ints((M, K), 9, 20).cuda(), _ints((M, N), 9, 23).cuda()
        want = m.mx4_linear(a, w.cuda(), s.cuda(), residual=res, mul=res)
        buf = res.clone()
        m.mx4_linear(a, w.cuda(), s.cuda(), residual=buf, mul=buf, out=buf)
        assert torch.equal(buf, want)
    with pytest.raises(ValueError, match="out overlaps residual"):
        big = torch.zeros((M + 1, N), dtype=BF16, device="cuda")
        m.mx4_linear(a, w.cuda(), s.cuda(), residual=big[1:], out=big[:M])


def test_rows_past_32_bit_offsets():
    """Output and operand offsets beyond 2^32 bytes and elements: the last rows of a long
    batch against the same rows alone, on tiles and widened."""
    from block_scaled_precision_amd import moe_mx as m
    N = 4096
    M = (1 << 32) // N + 1000
    for K in (512, 128):
        print_flush(f"mx4_linear 64-bit offsets M={M} K={K}")
        w, s = (t.cuda() for t in _codes((N,), K, 13))
        a = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")
        asc = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
        a[-40:] = _codes((40,), K, 13)[0].cuda()
        out = m.mx4_linear(a, w, s, a_scale=asc)
        assert torch.equal(out[-40:], m.mx4_linear(a[-40:].contiguous(), w, s, a_scale=asc[-40:].contiguous()))
        assert torch.equal(out[0], out[M - 41])
        del out, a, asc


@pytest.mark.parametrize("M,N", [(3, 24), (70, 264), (300, 520), (600, 4104)])
def test_longest_sum(M, N):
    """K = 2^24, where the 256 rows of a tile reach over 2^31 bytes: operands that are zero but
    for a few blocks (the last among them) give the products of those blocks alone."""
    from block_scaled_precision_amd import moe_mx as m
    K = 1 << 24
    print_flush(f"mx4_linear K=2^24 M={M} N={N}")
    blocks = [0, 5, 1 << 10, (1 << 18) + 3, (1 << 19) - 5, (1 << 19) - 4, (1 << 19) - 2, (1 << 19) - 1]
    (a8, s8), (w8, t8) = _codes((M,), 256, 17), _codes((N,), 256, 18)

    def spread(c, rows):
        full = torch.zeros((rows, K // 2), dtype=torch.uint8, device="cuda")
        for i, b in enumerate(blocks):
            full[:, 16 * b:16 * b + 16] = c[:, 16 * i:16 * i + 16].cuda()
        return full, torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")
    a, asc = spread(a8, M)
    w, wsc = spread(w8, N)
    ref, _, _ = mx4.mx4_linear(a8.numpy(), w8.numpy(), t8.numpy(), a_scale=s8.numpy())
    _same_bits(m.mx4_linear(a, w, wsc, a_scale=asc), ref, "longest sum")


AT_ONCE = [(100, 2056, 7168, 0, True), (5, 512, 1024, 0, False), (300, 2056, 640, 0, False), (700, 1032, 512, 4, True), (60, 4096, 1152, 0, False),
           (1500, 4104, 512, 5, False)]


def test_prepared_calls_at_once_and_captured():
    """Prepared calls of the same problem on two streams at the same time, then captured ones
    replayed among eager work: each has its own workspace."""
    from block_scaled_precision_amd import moe_mx as m
    for M, N, K, G, given in AT_ONCE:
        print_flush(f"mx4_linear at once M={M} N={N} K={K} G={G} codes {given}")
        w, s = (t.cuda() for t in _codes((G, N) if G else (N,), K, 19, scales=(118, 123)))
        off = torch.linspace(0, M, G + 1).int().cuda() if G else None
        a = [gen.normal((M, K), 19 + i, 25).to(BF16).cuda() for i in range(2)]
        a = [m.mx4_quantize(x) for x in a] if given else [(x, None) for x in a]
        want = [m.mx4_linear(x, w, s, a_scale=c, expert_offsets=off) for x, c in a]
        calls = [m.OpCall(m.mx4_linear, x, w, s, a_scale=c, expert_offsets=off) for x, c in a]
        streams = [torch.cuda.Stream() for _ in a]
        torch.cuda.synchronize()
        for _ in range(20):
            for call, st in zip(calls, streams):
                with torch.cuda.stream(st):
                    call()
        torch.cuda.synchronize()
        assert all(torch.equal(call(), r) for call, r in zip(calls, want))
        graphs = []
        for call in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = call()
            graphs.append((g, out))
        for i in (0, 1, 1, 0, 1):
            g, out = graphs[i]
            out.zero_()
            g.replay()
            other = m.mx4_linear(a[1 - i][0], w, s, a_scale=a[1 - i][1], expert_offsets=off)
            torch.cuda.synchronize()
            assert torch.equal(out, want[i]) and torch.equal(other, want[1 - i])


def _draw(n, seed=20261209):
    rng = np.random.default_rng(seed)
    out = []
    for i in range(n):
        G = int(rng.choice([0, 0, 1, 3, 9, 40]))
        M = int(np.exp(rng.uniform(0, np.log(3000))))
        N, K = 8 * int(np.exp(rng.uniform(0, np.log(300)))), 128 * int(rng.integers(1, 17))
        out.append(pytest.param(M, N, K, G, bool(rng.integers(2)), i))
    return out


@pytest.mark.parametrize("M,N,K,G,given,i", _draw(40))
def test_drawn_shapes_are_bit_identical(M, N, K, G, given, i):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear drawn M={M} N={N} K={K} G={G} codes {given}")
    rng = np.random.default_rng(i)
    w, s = _codes((G, N) if G else (N,), K, 14 + i)
    a, asc = _codes((M,), K, 40 + i) if given else (_ints((M, K), 14 + i, 20), None)
    bias, res = _ints((G, N) if G else (N,), 15 + i, 22, torch.float32), _ints((M, N), 16 + i, 23)
    offsets = np.concatenate([[0], np.sort(rng.integers(0, M + 1, G))]) if G else None
    ref, _, _ = mx4.mx4_linear(a.numpy() if given else _np(a), w.numpy(), s.numpy(),
                               a_scale=asc.numpy() if given else None, bias=_np(bias), residual=_np(res), offsets=offsets)
    off = None if offsets is None else torch.from_numpy(offsets).int().cuda()
    got = m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), a_scale=asc.cuda() if given else None, bias=bias.cuda(),
                       residual=res.cuda(), expert_offsets=off)
    _same_bits(got, ref, "drawn")


def test_a_linear_layer_trains_on_operands():
    """Forward, input and weight gradients of one projection as three products, rotated, the
    output's gradient rounded stochastically: each is the exact product of the operands'
    values to within the bound of a sum (dX, dW), and rotation leaves the mean relative error
    of a product of rows with outliers below that of the plain blocks."""
    from block_scaled_precision_amd import moe_mx as m
    T, N, K = 300, 264, 520
    x, wt, dy = gen.normal((T, K), 60, 1).to(BF16), gen.normal((N, K), 60, 2, std=0.02), gen.normal((T, N), 60, 3).to(BF16)
    x[:, ::97] *= 30
    signs = torch.where(gen.random_bytes((32,), 60, 4) < 128, -1.0, 1.0)
    rnd = gen.random_bytes((T, N), 60, 5)
    xc, wc, dc, sg, rg = x.cuda(), wt.cuda(), dy.cuda(), signs.cuda(), rnd.cuda()

    def product(a, b):
        (ac, asc), (bc, bsc) = a, b
        got = m.mx4_linear(ac, bc, bsc, a_scale=asc)
        av, bv = (_np(m.mx4_dequantize(*t, dtype=torch.float32)) for t in (a, b))
        ref, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
        bound = 2.0 ** -8 * np.abs(ref) + (1 + 2.0 ** -8) * 2 * av.shape[1] * 2.0 ** -24 * size
        assert (np.abs(_np(got) - ref) <= bound).all()
        return _np(got)
    q = m.mx4_quantize
    y = product(q(xc, signs=sg), q(wc, signs=sg))
    plain = product(q(xc), q(wc))
    exact = _np(x) @ _np(wt).T
    assert np.linalg.norm(y - exact) < np.linalg.norm(plain - exact)
    dx = product(q(dc, signs=sg, random=rg), q(wc, transpose=True, signs=sg))
    dw = product(q(dc, transpose=True, signs=sg, random=rg), q(xc, transpose=True, signs=sg))
    assert dx.shape == (T, K) and dw.shape == (N, K)
