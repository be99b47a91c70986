"""mx4_linear's large tiles against float64, on a sample of rows and columns: every row of a first
and of a ragged last tile and both sides of every group's ends, every column of a column block
and of the ragged last one, and others at random.

Bounds and exactness as in tests/test_gpu_mx4_linear.py.  The tiles' SiLU takes exp(-|v|) as t =
exp2(-|v| log2 e), off by |v| + 2 half steps of fp32: at most 16 of f = |v| t / (1 + t) up to |v|
= 14; past it f is below 1.2e-5 and the rest, (|v| + 2) E32 f < 1.3e-11, lies below the bound's dv
= 2 (K + 1) E32 (sum |a w| + |bias|) >= 2 K E32 |v|.
"""
import numpy as np
import pytest
import torch

import tests.test_gpu_mx4_linear as lin
from block_scaled_precision_amd import inputs as gen
from oracle import mx, mx4
from tests.conftest import has_gpu
from tests.helpers import print_flush
from tests.test_gpu_linear import BF16, _bound, _ints, _np
from tests.test_gpu_mx4_linear import CASES, _codes, _offsets

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

# (kernel, rows of its tiles, M, N, K, groups); tests/test_mx4_tiles_plan.py holds the lists of
# this file against the choice.  K: stages of 256 even and odd in number, the last one whole and
# half; fewer items than workgroups, and several for each.
LARGE = [
    ("tile", 128, 1500, 4104, 512, 0), ("tile", 128, 6000, 520, 640, 0), ("tile", 128, 6000, 520, 768, 0),
    ("tile", 128, 6000, 520, 896, 0), ("tile", 128, 9000, 4104, 640, 0), ("tile", 128, 6000, 520, 512, 1),
    ("tile", 128, 6000, 520, 768, 5), ("tile", 128, 8000, 264, 896, 40), ("tile", 128, 9300, 4104, 512, 3),
    ("tile", 256, 3000, 4104, 1920, 0), ("tile", 256, 3000, 4104, 2048, 0), ("tile", 256, 5000, 1544, 2176, 0),
    ("tile", 256, 5000, 1544, 2304, 0), ("tile", 256, 9300, 2568, 3200, 0), ("tile", 256, 5000, 1544, 2048, 1),
    ("tile", 256, 5000, 1544, 2304, 5), ("tile", 256, 6000, 1032, 1920, 40), ("tile", 256, 6000, 4104, 1664, 3),
    ("widen", 0, 3000, 1032, 128, 6), ("widen", 0, 1500, 520, 384, 0),
]
LARGE_IDS = [f"{k}{r}_{M}x{N}x{K}_g{G}" for k, r, M, N, K, G in LARGE]


def _sample(M, N, tile, off, seed):
    """Rows and columns to compare, ascending."""
    rng = np.random.default_rng(seed)
    tile = tile or 192
    ends = [0, M] if off is None else [int(e) for e in off]
    rows = {*range(min(tile, M)), *range((M - 1) // tile * tile, M), *rng.integers(0, M, 60).tolist()}
    rows |= {r for e in ends for r in (e - 1, e) if 0 <= r < M}
    block = 256 * int(rng.integers(0, max(N // 256, 1)))
    cols = {*range(block, min(block + 256, N)), *range((N - 1) // 256 * 256, N), *rng.integers(0, N, 60).tolist()}
    return np.array(sorted(rows)), np.array(sorted(cols))


def _sampled_offsets(rows, off):
    return None if off is None else np.searchsorted(rows, off)


def _fn64(v, fn):
    x = torch.from_numpy(v)
    if fn == "silu":
        return (x / (1 + torch.exp(-x))).numpy()
    if fn == "gelu":
        return (x * torch.special.erfc(-x / 2 ** 0.5) / 2).numpy()
    return np.maximum(v, 0) ** 2 if fn == "relu2" else v


@pytest.mark.parametrize("fn", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("kernel,tile,M,N,K,G", LARGE, ids=LARGE_IDS)
def test_functions_factors_and_residuals(kernel, tile, M, N, K, G, fn):
    """Every function with a bias of either type or none, a second factor, a residual, both."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear {fn} {kernel}{tile} M={M} N={N} K={K} G={G}")
    a = gen.normal((M, K), 4, 25).to(BF16)
    shape = (G, N) if G else (N,)
    w, s = _codes(shape, K, 4, scales=(118, 123))
    bias = gen.normal(shape, 4, 26)
    mul, res = gen.normal((M, N), 4, 27).to(BF16), gen.normal((M, N), 4, 28).to(BF16)
    off = _offsets(M, G, M + N)
    rows, cols = _sample(M, N, tile, off, M)
    part = _sampled_offsets(rows, off)
    pick = np.ix_(rows, cols)
    wn, sn = (t.numpy()[:, cols] if G else t.numpy()[cols] for t in (w, s))
    v0, size, _ = mx4.mx4_linear(_np(a[rows]), wn, sn, offsets=part)
    kw = dict(fn=fn, expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    a, w, s = a.cuda(), w.cuda(), s.cuda()
    for b, mu, re in ((None, None, None), (bias, None, None), (bias.to(BF16), mul, None), (None, None, res),
                      (bias, mul, res), (None, mul, res)):
        got = m.mx4_linear(a, w, s, bias=None if b is None else b.cuda(), mul=None if mu is None else mu.cuda(),
                           residual=None if re is None else re.cuda(), **kw)
        assert torch.isfinite(got).all()
        b64 = np.zeros((len(rows), len(cols)))
        if b is not None:
            b64 += np.repeat(_np(b)[:, cols], np.diff(part), axis=0) if G else _np(b)[cols]
        mu64, re64 = (1.0 if mu is None else _np(mu)[pick]), (0.0 if re is None else _np(re)[pick])
        ref = _fn64(v0 + b64, fn) * mu64 + re64
        d = np.abs(_np(got.cpu()[pick]) - ref)
        bound = _bound(fn, K, v0 + b64, size, b64, mu64, re64, ref)
        assert (d <= bound).all(), f"{(d > bound).sum()} out of bounds, worst ratio {(d / bound).max():.2f}"


ALL = CASES + [c for c in LARGE if c not in CASES]


@pytest.mark.parametrize("kernel,tile,M,N,K,G", ALL, ids=[f"{k}{r}_{M}x{N}x{K}_g{G}" for k, r, M, N, K, G in ALL])
def test_fp32_bias_and_relu2_are_bit_identical(kernel, tile, M, N, K, G):
    """Results below 2^20 (|v| < 2^10 is a multiple of 1/4: its square has 24 bits), compared
    one by one; K = 16384, whose v has a standard deviation of 1096, leaves 65 % of them."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_linear relu2 {kernel}{tile} M={M} N={N} K={K} G={G}")
    shape = (G, N) if G else (N,)
    (a, asc), (w, s), bias = _codes((M,), K, 0), _codes(shape, K, 1), _ints(shape, 1, 22, torch.float32)
    off = _offsets(M, G, M + N)
    rows, cols = _sample(M, N, tile, off, M)
    wn, sn, bn = (t.numpy()[:, cols] if G else t.numpy()[cols] for t in (w, s, bias))
    ref, _, _ = mx4.mx4_linear(a.numpy()[rows], wn, sn, a_scale=asc.numpy()[rows], offsets=_sampled_offsets(rows, off),
                               bias=bn.astype(np.float64), fn="relu2")
    got = m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), a_scale=asc.cuda(), bias=bias.cuda(), fn="relu2",
                       expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    got = _np(got.cpu()[np.ix_(rows, cols)])
    exact = ref < 2.0 ** 20
    # (half of the values are negative, results 0: positive ones have to be among the compared)
    assert exact.mean() > 0.5 and (ref[exact] > 0).mean() > (0.1 if ref.size > 1000 else 0)
    bad = np.argwhere(exact & (got != mx.round_to_bf16(ref)))
    assert bad.size == 0, f"{len(bad)} of {exact.sum()} differ, first at {rows[bad[0][0]], cols[bad[0][1]]}"


# (M, N, K) of 256-row tiles, without groups and with 5
SCALED = [(3000, 4104, 1920), (3000, 4104, 2048), (5000, 1544, 2176), (5000, 1544, 2304)]


@pytest.mark.parametrize("G", [0, 5])
@pytest.mark.parametrize("M,N,K", SCALED)
def test_every_code_meets_its_scales(M, N, K, G):
    lin.test_every_code_meets_its_scales(M, N, K, G)


@pytest.mark.parametrize("M,N,K", SCALED)
def test_nan_scales_and_infinite_results(M, N, K):
    lin.test_nan_scales_and_infinite_results(M, N, K)


# (N, K, rows of each group), 256-row tiles: ends at, before and behind a tile's and a wave's
COUNTS = [(1544, 1664, (256, 257, 255, 0, 1, 512, 3000, 719)), (1544, 2304, (0, 33, 4000, 95, 0, 1000)),
          (4104, 1920, (2900,))]


@pytest.mark.parametrize("N,K,counts", COUNTS, ids=str)
def test_groups_are_bit_identical(N, K, counts):
    lin.test_groups_are_bit_identical(N, K, list(counts))


OUT_OF_ORDER = [(5000, 1544, 1664)]  # 4 groups


@pytest.mark.parametrize("M,N,K", OUT_OF_ORDER)
def test_offsets_out_of_order_or_range_stay_in_bounds(M, N, K):
    from block_scaled_precision_amd import moe_mx as m
    lin.test_offsets_out_of_order_or_range_stay_in_bounds(M, N, K)
    a, (w, s) = _ints((M, K), 8, 20), _codes((4, N), K, 8)
    buf = torch.full((3 * M, N), 9.0, dtype=BF16, device="cuda")
    for off in ([0, M, 5, M, 80], [0, 1000, 3000, 5000, 10 ** 6], [-2 ** 31, 2 ** 31 - 1, 0, 5, 9]):
        m.mx4_linear(a.cuda(), w.cuda(), s.cuda(), expert_offsets=torch.tensor(off, dtype=torch.int32).cuda(),
                     out=buf[M:2 * M])
        torch.cuda.synchronize()
        assert (buf[:M] == 9.0).all() and (buf[2 * M:] == 9.0).all()


ALIGNED = [(3000, 4104, 1920, 0), (5000, 1544, 2304, 5), (6000, 4104, 1664, 3)]


@pytest.mark.parametrize("M,N,K,G", ALIGNED)
def test_biases_of_any_alignment(M, N, K, G):
    """Either type, from every address of the type; the bias differs in every column and group,
    and NaN stands before and behind it."""
    from block_scaled_precision_amd import moe_mx as m
    shape = (G, N) if G else (N,)
    (w, s), (a, asc) = _codes(shape, K, 50), _codes((M,), K, 51)
    off = _offsets(M, G, M)
    rows, cols = _sample(M, N, 256, off, M)
    wn, sn = (t.numpy()[:, cols] if G else t.numpy()[cols] for t in (w, s))
    v, _, _ = mx4.mx4_linear(a.numpy()[rows], wn, sn, a_scale=asc.numpy()[rows], offsets=_sampled_offsets(rows, off))
    kw = dict(a_scale=asc.cuda(), expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    a, w, s, n = a.cuda(), w.cuda(), s.cuda(), max(G, 1) * N
    values = ((torch.arange(n) * 37) % 509 - 254).float()
    for dtype, step in ((torch.float32, 4), (BF16, 2)):
        b = _np(values.to(dtype)).reshape(shape)
        ref = v + (np.repeat(b[:, cols], np.diff(_sampled_offsets(rows, off)), axis=0) if G else b[cols])
        for at in range(0, 16, step):
            buf = torch.full((n + 16,), float("nan"), dtype=dtype, device="cuda")
            view = buf[at // step:at // step + n]
            view.copy_(values)
            got = m.mx4_linear(a, w, s, bias=view.view(shape), **kw).cpu()
            assert np.array_equal(_np(got[np.ix_(rows, cols)]), mx.round_to_bf16(ref)), f"{dtype} at {at}"


IN_PLACE = [(9300, 2568, 3200, 0), (6000, 4104, 1664, 3), (9000, 4104, 640, 0)]


@pytest.mark.parametrize("M,N,K,G", IN_PLACE)
def test_out_may_be_factor_and_residual(M, N, K, G):
    from block_scaled_precision_amd import moe_mx as m
    w, s = (t.cuda() for t in _codes((G, N) if G else (N,), K, 9))
    a, asc = (t.cuda() for t in _codes((M,), K, 10))
    res = _ints((M, N), 9, 23).cuda()
    off = _offsets(M, G, M)
    kw = dict(a_scale=asc, expert_offsets=None if off is None else torch.from_numpy(off).int().cuda())
    want = m.mx4_linear(a, w, s, residual=res, mul=res, **kw)
    buf = res.clone()
    m.mx4_linear(a, w, s, residual=buf, mul=buf, out=buf, **kw)
    assert torch.equal(buf, want)


# (M, N, K, groups, codes given)
AT_ONCE = [(3000, 4104, 1920, 0, True), (5000, 1544, 2304, 5, False), (9300, 2568, 3200, 0, False), (9000, 4104, 640, 0, True)]


def test_prepared_calls_at_once_and_captured(monkeypatch):
    monkeypatch.setattr(lin, "AT_ONCE", AT_ONCE)
    lin.test_prepared_calls_at_once_and_captured()


@pytest.mark.parametrize("M,N,K", [(16, 256, 128), (255, 256, 7168), (700, 1032, 128), (700, 1032, 1152), (1500, 4104, 512),
                                   (3000, 4104, 1920)])
def test_every_pair_of_scales(M, N, K):
    """1 times 1 at the first and the last k, with every scale of a row against every scale of a
    column: 2^-254 to 2^254, of which bf16 holds 2^-133 (a subnormal) to 2^127; from half of
    its smallest number down they are 0, above its range infinite."""
    from block_scaled_precision_amd import moe_mx as m
    ra, rw = torch.arange(M) % 255, torch.arange(N) % 255
    e = (ra[:, None] + rw - 254).numpy()
    for k in (0, K - 1):
        (a, asc), (w, wsc) = _codes((M,), K, 70), _codes((N,), K, 71)
        for t, s, r in ((a, asc, ra), (w, wsc, rw)):
            t.zero_()
            t[:, k // 2] = 2 << 4 * (k % 2)
            s[:, k // 32] = r.to(torch.uint8)
        got = _np(m.mx4_linear(a.cuda(), w.cuda(), wsc.cuda(), a_scale=asc.cuda()))
        want = np.where(e > 127, np.inf, np.where(e < -133, 0.0, np.ldexp(1.0, e)))
        assert np.array_equal(got, want)
