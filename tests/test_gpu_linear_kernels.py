"""mx_linear on every kernel it can choose, against a plain computation in 64 bits.

CASES names the kernel each shape is meant for; tests/test_linear_plan.py checks on
the host that the choice agrees and that no kernel, weight format, activation type or
grouping goes without a case.  The large-tile kernels (mid, tiled, wide) have shapes
whose items outnumber the workgroups, column blocks that N cuts (N % 256 != 0) and,
where the kernel takes them, K off its scale groups (K % 512 != 0).

Bounds, with e = 2^-24 and u = 2^-8 (half a step of bf16): an fp32 sum of K products
and the bias, in any order and with truncating additions, is off by at most dv = 2 (K
+ 1) e (sum |a w| + |bias|).  A function moves by its slope (|silu'| <= 1.1, |gelu'| <=
1.13, relu2' = 2 max(v, 0)) times dv, and computes within 16 e of its value; GELU's
exp(-v^2 / 2) adds v^2 e from its rounded argument on either side, and its polynomial
stays within 16 e as well.  Below |v| = 13.2 the exponential is a normal number; past
it the result is below 2^-123 and may be 0.  mul, residual and the output rounding
follow term by term.
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from oracle import gemm as og
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

BITS = {"e2m1": 4, "e3m2": 6}
E32, U = 2.0 ** -24, 2.0 ** -8
BF16 = torch.bfloat16

# (kernel, tile rows, K ranges at all, M, N, K, groups, fmt, act)
CASES = [
    ("few", 16, False, 9, 264, 128, 0, "e2m1", "bf16"),
    ("rows", 16, False, 5, 8200, 128, 0, "e2m1", "bf16"),
    ("rows", 16, True, 17, 264, 7168, 0, "e2m1", "bf16"),
    ("rows", 64, False, 2900, 264, 128, 0, "e2m1", "bf16"),
    ("rows", 64, True, 520, 264, 7168, 0, "e2m1", "bf16"),
    ("mid", 64, False, 6100, 264, 512, 0, "e2m1", "bf16"),
    ("mid", 64, False, 900, 8200, 896, 0, "e2m1", "bf16"),
    ("mid", 128, False, 2900, 2056, 512, 0, "e2m1", "bf16"),
    ("mid", 128, False, 20000, 520, 640, 0, "e2m1", "bf16"),
    ("few", 16, False, 9, 264, 128, 0, "e2m1", "mxfp8"),
    ("rows", 16, False, 1, 8200, 128, 0, "e2m1", "mxfp8"),
    ("rows", 16, True, 1, 8200, 3712, 0, "e2m1", "mxfp8"),
    ("rows", 64, False, 1540, 264, 128, 0, "e2m1", "mxfp8"),
    ("rows", 64, True, 17, 4104, 7168, 0, "e2m1", "mxfp8"),
    ("tiled", 128, False, 2900, 2056, 640, 0, "e2m1", "mxfp8"),
    ("tiled", 128, False, 20000, 520, 512, 0, "e2m1", "mxfp8"),
    ("tiled", 192, False, 1000, 4104, 640, 0, "e2m1", "mxfp8"),
    ("tiled", 192, False, 30000, 264, 640, 0, "e2m1", "mxfp8"),
    ("wide", 192, False, 2100, 4160, 1024, 0, "e2m1", "mxfp8"),
    ("wide", 192, False, 30000, 576, 1024, 0, "e2m1", "mxfp8"),
    ("few", 16, False, 9, 264, 128, 0, "e3m2", "bf16"),
    ("rows", 16, False, 5, 8200, 128, 0, "e3m2", "bf16"),
    ("rows", 16, True, 17, 264, 7168, 0, "e3m2", "bf16"),
    ("rows", 64, False, 1540, 264, 128, 0, "e3m2", "bf16"),
    ("rows", 64, True, 200, 520, 7168, 0, "e3m2", "bf16"),
    ("few", 16, False, 9, 264, 128, 0, "e3m2", "mxfp8"),
    ("rows", 16, False, 1, 8200, 128, 0, "e3m2", "mxfp8"),
    ("rows", 16, True, 1, 8200, 3712, 0, "e3m2", "mxfp8"),
    ("rows", 64, False, 1540, 264, 128, 0, "e3m2", "mxfp8"),
    ("rows", 64, True, 520, 264, 7168, 0, "e3m2", "mxfp8"),
    ("tiled", 128, False, 2900, 2056, 640, 0, "e3m2", "mxfp8"),
    ("tiled", 128, False, 20000, 520, 640, 0, "e3m2", "mxfp8"),
    ("tiled", 192, False, 1000, 4104, 640, 0, "e3m2", "mxfp8"),
    ("tiled", 192, False, 30000, 264, 512, 0, "e3m2", "mxfp8"),
    ("few", 16, False, 12, 264, 128, 5, "e2m1", "bf16"),
    ("rows", 16, False, 12, 8200, 128, 5, "e2m1", "bf16"),
    ("rows", 64, False, 2900, 264, 128, 5, "e2m1", "bf16"),
    ("mid", 64, False, 4500, 1544, 640, 5, "e2m1", "bf16"),
    ("mid", 128, False, 20000, 520, 640, 5, "e2m1", "bf16"),
    ("few", 16, False, 12, 264, 128, 5, "e2m1", "mxfp8"),
    ("rows", 16, False, 12, 8200, 128, 5, "e2m1", "mxfp8"),
    ("rows", 64, False, 1540, 264, 128, 5, "e2m1", "mxfp8"),
    ("tiled", 128, False, 20000, 520, 640, 5, "e2m1", "mxfp8"),
    ("tiled", 192, False, 900, 8200, 512, 5, "e2m1", "mxfp8"),
    ("tiled", 192, False, 30000, 264, 640, 5, "e2m1", "mxfp8"),
    ("wide", 192, False, 1900, 8256, 1024, 5, "e2m1", "mxfp8"),
    ("few", 16, False, 12, 264, 128, 5, "e3m2", "bf16"),
    ("rows", 16, False, 12, 8200, 128, 5, "e3m2", "bf16"),
    ("rows", 64, False, 1540, 264, 128, 5, "e3m2", "bf16"),
    ("few", 16, False, 12, 264, 128, 5, "e3m2", "mxfp8"),
    ("rows", 16, False, 12, 8200, 128, 5, "e3m2", "mxfp8"),
    ("rows", 64, False, 1540, 264, 128, 5, "e3m2", "mxfp8"),
    ("tiled", 128, False, 20000, 520, 640, 5, "e3m2", "mxfp8"),
    ("tiled", 192, False, 900, 8200, 512, 5, "e3m2", "mxfp8"),
]
_NAMES = [f"{k}{r}{'_split' if s else ''}_{M}x{N}x{K}_G{G}_{f}_{a}" for k, r, s, M, N, K, G, f, a in CASES]
SHAPES = pytest.mark.parametrize("M,N,K,G,fmt,act", [c[3:] for c in CASES], ids=_NAMES)
# of each kernel with a tile list or K ranges, the case with the most of them
LARGE = [c[3:] for c in CASES if c[0] in ("mid", "tiled", "wide") or c[2]]
LARGE_IDS = [n for n, c in zip(_NAMES, CASES) if c[0] in ("mid", "tiled", "wide") or c[2]]


def _offsets(M, G):
    """G groups over M - 3 rows: empty ones first and in the middle, one of one row,
    the rest uneven; offsets start at 7."""
    P = M - 3
    third = 1 + (P - 1) // 3
    return [7 + n for n in (0, 0, 1, third, third, P)], P


def _weights(G, N, K, fmt, seed, scales=None):
    """Codes and scales [G or 1, N, ...] (codes 127: scales of 1)."""
    w = gen.random_bytes((max(G, 1), N, K * BITS[fmt] // 8), seed, 21)
    if scales is None:
        return w, torch.full((max(G, 1), N, K // 32), 127, dtype=torch.uint8)
    g = torch.Generator().manual_seed(seed)
    return w, torch.randint(*scales, (max(G, 1), N, K // 32), generator=g, dtype=torch.uint8)


def _decoded(w, s, fmt, K):
    return [torch.from_numpy(og.decode_weight(w[g].numpy(), s[g].numpy(), fmt, K)).cuda() for g in range(len(w))]


def _product(a, act, W, offsets, P, size=False):
    """v [P, N] (and the sums of magnitudes) in float64 on the GPU."""
    A = torch.from_numpy(og.activations(a[:P].double().numpy(), act)).cuda()
    v = torch.empty((P, W[0].shape[0]), dtype=torch.float64, device="cuda")
    m = torch.empty_like(v) if size else None
    for g, Wg in enumerate(W):
        lo, hi = (0, P) if offsets is None else (offsets[g] - offsets[0], offsets[g + 1] - offsets[0])
        if lo < hi:
            v[lo:hi] = A[lo:hi] @ Wg.t().contiguous()
            if size:
                m[lo:hi] = A[lo:hi].abs() @ Wg.abs().t().contiguous()
    return (v, m) if size else v


def _per_row(bias, offsets, P):
    """bias [G, N] as the rows see it, float64."""
    if offsets is None:
        return bias[0].double()[None]
    counts = torch.tensor([b - a for a, b in zip(offsets[:-1], offsets[1:])])
    return bias.double().repeat_interleave(counts.to(bias.device), 0)


def _problem(M, N, K, G, fmt, act, seed, scales=None):
    offsets, P = _offsets(M, G) if G else (None, M)
    w, s = _weights(G, N, K, fmt, seed, scales)
    wd, sd = (w.cuda(), s.cuda()) if G else (w[0].cuda(), s[0].cuda())
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    return offsets, P, w, s, wd, sd, off


@SHAPES
def test_exact_products_are_bit_identical(M, N, K, G, fmt, act):
    """Small integers and weights of scale 1: every sum is a multiple of 1/16 within
    24 bits, so v + bias, times a power of two or plus an integer, is exact and its
    one rounding has to agree bit for bit."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: exact M={M} N={N} K={K} G={G} {fmt}/{act}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 30)
    a = gen.small_integers((M, K), 30, 20).to(BF16)
    v = _product(a, act, _decoded(w, s, fmt, K), offsets, P)
    a[P:] = float("nan")  # rows behind the last group
    ad = a.cuda()

    def check(out, ref, what):
        bad = torch.nonzero(out[:P] != ref.to(BF16))
        assert len(bad) == 0, f"{what}: {len(bad)} of {P * N} differ, first at {bad[0].tolist()}"
        assert (out[P:] == 33.0).all(), f"{what}: rows behind the last group"

    out = torch.full((M, N), 33.0, dtype=BF16, device="cuda")
    m.mx_linear(ad, wd, sd, fmt, act, expert_offsets=off, out=out)
    check(out, v, "plain")
    bias = gen.small_integers((max(G, 1), N), 31, 22).float().cuda()
    res = gen.small_integers((M, N), 32, 23).to(BF16).cuda()
    res[P:] = 33.0
    vb = v + _per_row(bias, offsets, P)
    shifted = torch.cat([bias.new_zeros(1), bias.view(-1)])[1:].view(bias.shape)  # off 16-byte addresses
    for b in (bias, bias.to(BF16), shifted, torch.cat([bias.new_zeros(1), bias.view(-1)]).to(BF16)[1:].view(bias.shape)):
        buf = res.clone()
        m.mx_linear(ad, wd, sd, fmt, act, bias=b if G else b[0], residual=buf, expert_offsets=off, out=buf)
        check(buf, vb + res[:P].double(), "bias, residual in place")
    mul = (2.0 ** gen.small_integers((M, N), 33, 24, -2, 2).float()).to(BF16).cuda()
    mul[P:] = 33.0
    m.mx_linear(ad, wd, sd, fmt, act, bias=bias if G else bias[0], mul=mul, expert_offsets=off, out=mul)
    powers = 2.0 ** gen.small_integers((M, N), 33, 24, -2, 2).double().cuda()
    check(mul, vb * powers[:P], "bias, mul in place")


def _fn(v, fn):
    if fn == "none":
        return v
    if fn == "silu":
        return v * torch.sigmoid(v)
    if fn == "gelu":
        return 0.5 * v * torch.special.erfc(-v * 0.5 ** 0.5)
    return v.clamp(min=0) ** 2


def _fn_bound(v, f, dv, fn):
    if fn == "none":
        return dv
    if fn == "silu":
        return 1.1 * dv + 16 * E32 * (f.abs() + dv)
    if fn == "gelu":
        return 1.13 * dv + (16 + 2 * v * v) * E32 * (f.abs() + dv) + E32 * v.abs() * E32 + 2.0 ** -123
    return (2 * v.abs() + dv) * dv + 4 * E32 * (f.abs() + dv)


@pytest.mark.parametrize("M,N,K,G,fmt,act", LARGE, ids=LARGE_IDS)
def test_functions_within_their_bound(M, N, K, G, fmt, act):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: functions M={M} N={N} K={K} G={G} {fmt}/{act}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 34, scales=(116, 121))
    a = gen.normal((M, K), 34, 25).to(BF16)
    bias = gen.normal((max(G, 1), N), 34, 26).cuda()
    v, size = _product(a, act, _decoded(w, s, fmt, K), offsets, P, size=True)
    b = _per_row(bias, offsets, P)
    v = v + b
    dv = 2 * (K + 1) * E32 * (size + b.abs())
    mul, res = (gen.normal((M, N), 34, i).to(BF16).cuda() for i in (27, 28))
    for fn in ("none", "silu", "gelu", "relu2"):
        f = _fn(v, fn)
        df = _fn_bound(v, f, dv, fn)
        for mu, re in ((None, None), (mul, res)):
            out = m.mx_linear(a.cuda(), wd, sd, fmt, act, bias=bias if G else bias[0], fn=fn, mul=mu, residual=re,
                              expert_offsets=off)[:P].double()
            mu64 = 1.0 if mu is None else mu[:P].double()
            re64 = 0.0 if re is None else re[:P].double()
            ref = f * mu64 + re64
            d = df * abs(mu64) * (1 + 2 * E32) + 2 * E32 * ((f * mu64).abs() + abs(re64))
            bound = U * ref.abs() + (1 + U) * d
            worst = ((out - ref).abs() / bound.clamp(min=1e-300)).max().item()
            assert worst <= 1.0, f"{fn}: worst ratio {worst:.3f}"


@SHAPES
def test_every_weight_meets_its_scale(M, N, K, G, fmt, act):
    """Row m holds one nonzero power of two, at k = 33 m mod K: out[m, n] is a weight
    times its block's scale and that power, exactly."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: scales M={M} N={N} K={K} G={G} {fmt}/{act}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 35, scales=(60, 190))
    rows, k = torch.arange(M), 33 * torch.arange(M) % K
    power = 2.0 ** (rows % 9 - 4).double()
    a = torch.zeros((M, K), dtype=BF16)
    a[rows, k] = power.to(BF16)
    out = m.mx_linear(a.cuda(), wd, sd, fmt, act, expert_offsets=off)
    for g, W in enumerate(_decoded(w, s, fmt, K)):
        lo, hi = (0, P) if offsets is None else (offsets[g] - offsets[0], offsets[g + 1] - offsets[0])
        ref = W[:, k[lo:hi].cuda()].t() * power[lo:hi, None].cuda()
        assert torch.equal(out[lo:hi].double(), ref), f"group {g}"


@pytest.mark.parametrize("M,N,K,G,fmt,act", [c for c in LARGE if c[3]],
                         ids=[n for n, c in zip(LARGE_IDS, LARGE) if c[3]])
def test_offsets_out_of_order_or_range_stay_in_bounds(M, N, K, G, fmt, act):
    """Whatever the offsets hold, the tile list stays inside its room and nothing
    outside [M, N] is written."""
    from block_scaled_precision_amd import moe_mx as m
    _, _, _, _, wd, sd, _ = _problem(M, N, K, G, fmt, act, 36)
    a = gen.small_integers((M, K), 36, 20).to(BF16).cuda()
    guard = 64
    buf = torch.full((M + 2 * guard, N), 9.0, dtype=BF16, device="cuda")
    need = m.lib().mx_linear_workspace_bytes(m.MxLinearProblem(M, N, K, G, m.ACTS[act], m.MX_FORMATS[fmt], 0, 0, 0, 0), 0)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for off in ([0, 10 * M, 5, M // 2, 3 * M, 1], [7, 3, 2, 1, 0, -9], [-2 ** 31, 2 ** 31 - 1, 0, 5, 9, 2 ** 31 - 1],
                [0, M, M, M // 3, M, M]):
        print_flush(f"mx_linear kernels: offsets {off} M={M} N={N} K={K} {fmt}/{act}")
        m.mx_linear(a, wd, sd, fmt, act, expert_offsets=torch.tensor(off, dtype=torch.int32, device="cuda"),
                    out=buf[guard:guard + M], workspace=ws[:need])
        torch.cuda.synchronize()
        assert (buf[:guard] == 9.0).all() and (buf[guard + M:] == 9.0).all()
        assert (ws[need:] == 0xA5).all()


@pytest.mark.parametrize("M,N,K,G,fmt,act", LARGE, ids=LARGE_IDS)
def test_prepared_calls_at_once_and_captured(M, N, K, G, fmt, act):
    """Two prepared calls with a whole epilogue on two streams at the same time, then
    captured and replayed in turn among eager work: each has its own workspace (tile
    list, partial sums, quantized rows)."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: at once M={M} N={N} K={K} G={G} {fmt}/{act}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 37, scales=(116, 121))
    a = [gen.normal((M, K), 37 + i, 25).to(BF16).cuda() for i in range(2)]
    mul, res = (gen.normal((M, N), 37, i).to(BF16).cuda() for i in (27, 28))
    bias = gen.normal((max(G, 1), N), 37, 26).cuda()
    kw = dict(bias=bias if G else bias[0], fn="silu", mul=mul, residual=res, expert_offsets=off)
    want = [m.mx_linear(x, wd, sd, fmt, act, **kw)[:P].clone() for x in a]
    assert not torch.equal(want[0], want[1])
    calls = [m.OpCall(m.mx_linear, x, wd, sd, fmt, act, **kw) for x in a]
    streams = [torch.cuda.Stream() for _ in a]
    torch.cuda.synchronize()
    for _ in range(8):
        for call, st in zip(calls, streams):
            with torch.cuda.stream(st):
                call()
    torch.cuda.synchronize()
    graphs = []
    for call, r in zip(calls, want):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        assert torch.equal(out[:P], r)
        graphs.append((g, out))
    for i in (0, 1, 1, 0, 1):
        g, out = graphs[i]
        out.zero_()
        g.replay()
        other = m.mx_linear(a[1 - i], wd, sd, fmt, act, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out[:P], want[i]) and torch.equal(other[:P], want[1 - i])


def test_many_rows_of_few_columns():
    """Eight columns and more rows than the few-row kernel's launch can have: the last
    rows against the same rows alone."""
    from block_scaled_precision_amd import moe_mx as m
    M, N, K = (1 << 24) + 100, 8, 128
    print_flush(f"mx_linear kernels: M={M} N={N} K={K}")
    w, s = _weights(0, N, K, "e2m1", 38)
    a = torch.ones((M, K), dtype=BF16, device="cuda")
    a[-40:] = gen.small_integers((40, K), 38, 20).to(BF16).cuda()
    out = m.mx_linear(a, w[0].cuda(), s[0].cuda(), "e2m1", "bf16")
    assert torch.equal(out[-40:], m.mx_linear(a[-40:].contiguous(), w[0].cuda(), s[0].cuda(), "e2m1", "bf16"))
    assert (out[:-40] == out[0]).all()


@pytest.mark.parametrize("fn", ["none", "silu", "gelu", "relu2"])
@pytest.mark.parametrize("M,N,K,G,fmt,act", [c[3:] for c in CASES if c[8] == "bf16"],
                         ids=[n for n, c in zip(_NAMES, CASES) if c[8] == "bf16"])
def test_nan_and_infinity_arrive(M, N, K, G, fmt, act, fn):
    """A NaN in one row of A makes that row of out NaN whatever the function, a bias of
    infinity its column infinite; the rest is as without them."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: NaN {fn} M={M} N={N} K={K} G={G} {fmt}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 39, scales=(116, 121))
    a = gen.normal((M, K), 39, 25).to(BF16).cuda()
    bias = gen.normal((max(G, 1), N), 39, 26).cuda()
    call = lambda: m.mx_linear(a, wd, sd, fmt, act, bias=bias if G else bias[0], fn=fn, expert_offsets=off)[:P].clone()
    plain = call()
    row, col = P // 2, N - 3
    a[row, K - 1] = float("nan")
    bias[:, col] = float("inf")
    out = call()
    assert torch.isnan(out[row]).all()
    keep = torch.ones(P, dtype=torch.bool, device="cuda")
    keep[row] = False
    assert (out[keep, col] == float("inf")).all()
    plain[:, col] = float("inf")
    assert torch.equal(out[keep], plain[keep])


# (kernel, M, N, K, groups, fmt, act): outputs of more than 2^32 values, or activations
# of more than 2^32 bytes; for wide, whose offsets into them have 32 bits, just fewer
LONG = [
    ("mid", (1 << 32) // 4104 + 1000, 4104, 512, 0, "e2m1", "bf16"),
    ("mid", (1 << 32) // 4104 + 1000, 4104, 512, 5, "e2m1", "bf16"),
    ("rows", (1 << 31) // 1024 + 1000, 264, 1024, 0, "e2m1", "bf16"),
    ("rows", (1 << 31) // 1024 + 1000, 264, 1024, 5, "e3m2", "bf16"),
    ("tiled", (1 << 32) // 4104 + 1000, 4104, 512, 0, "e3m2", "mxfp8"),
    ("tiled", (1 << 32) // 1024 + 1000, 264, 1024, 0, "e2m1", "mxfp8"),
    ("tiled", (1 << 32) // 1024 + 1000, 264, 1024, 5, "e3m2", "mxfp8"),
    ("wide", (1 << 32) // 4096 - 100, 4160, 4096, 0, "e2m1", "mxfp8"),
    ("wide", (1 << 32) // 4160 + 1000, 4160, 1024, 5, "e2m1", "mxfp8"),
    ("tiled", (1 << 32) // 4096 + 100, 4160, 4096, 0, "e2m1", "mxfp8"),
]


@pytest.mark.parametrize("kernel,M,N,K,G,fmt,act", LONG, ids=[f"{c[0]}_{c[1]}x{c[2]}x{c[3]}_G{c[4]}_{c[5]}_{c[6]}" for c in LONG])
def test_long_batches(kernel, M, N, K, G, fmt, act):
    """Rows of ones, the last 40 of small integers: those against the same rows alone,
    the others against the first of their group.  Every sum is exact."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: long {kernel} M={M} N={N} K={K} G={G} {fmt}/{act}")
    offsets, P, w, s, wd, sd, off = _problem(M, N, K, G, fmt, act, 40)
    tail = gen.small_integers((40, K), 40, 20).to(BF16).cuda()
    a = torch.ones((M, K), dtype=BF16, device="cuda")
    a[P - 40:P] = tail
    out = m.mx_linear(a, wd, sd, fmt, act, expert_offsets=off)
    last = (wd[G - 1], sd[G - 1]) if G else (wd, sd)
    assert torch.equal(out[P - 40:P], m.mx_linear(tail, *last, fmt, act))
    bounds = [0, P] if offsets is None else [o - offsets[0] for o in offsets]
    for g, (lo, hi) in enumerate(zip(bounds[:-1], bounds[1:])):
        hi = min(hi, P - 40)
        if lo < hi:
            one = m.mx_linear(a[:1], *((wd[g], sd[g]) if G else (wd, sd)), fmt, act)
            for i in range(lo, hi, 1 << 18):
                assert (out[i:min(hi, i + (1 << 18))] == one).all(), f"group {g}, rows from {i}"


@pytest.mark.parametrize("M,N,K,G,fmt,act", LARGE, ids=LARGE_IDS)
def test_halves_slices_and_codes(M, N, K, G, fmt, act):
    """The up half of [gate; up] weights, offsets that are a slice of a longer table,
    and activations given as codes and scales: the same bits as copies and bf16 rows."""
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx_linear kernels: halves and codes M={M} N={N} K={K} G={G} {fmt}/{act}")
    _, P, _, _, wd, sd, off = _problem(M, 2 * N, K, G, fmt, act, 41, scales=(116, 121))
    a = gen.normal((M, K), 41, 25).to(BF16).cuda()
    wu, su = wd[..., N:, :], sd[..., N:, :]
    want = m.mx_linear(a, wu.contiguous(), su.contiguous(), fmt, act, fn="gelu", expert_offsets=off)[:P]
    kw = dict(fn="gelu")
    if G:
        kw["expert_offsets"] = torch.cat([off.new_tensor([0, 3, 5]), off, off.new_tensor([M + 9])])[3:4 + G]
    assert torch.equal(m.mx_linear(a, wu, su, fmt, act, **kw)[:P], want)
    if act == "mxfp8":
        codes, scales = m.mx_quantize(a, "e4m3")
        assert torch.equal(m.mx_linear(codes, wu, su, fmt, act, a_scale=scales, **kw)[:P], want)
