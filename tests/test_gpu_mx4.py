"""mx4_quantize and mx4_dequantize on the GPU against the oracle: bit-exact codes, scales
and values."""
import numpy as np
import pytest
import torch

from block_scaled_precision_amd import inputs as gen
from oracle import mx4
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

F32, BF16 = torch.float32, torch.bfloat16
MODES = [(t, s, r) for t in (False, True) for s in (False, True) for r in (False, True)]


def _signs(seed):
    return torch.where(gen.random_bytes((32,), seed, 81) < 128, -1.0, 1.0)


def _wide_range(shape, seed):
    """Rows and values of many binades."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randint(-30, 30, (*shape[:-1], 1), generator=g).float())
    return x * torch.exp2(torch.randint(-8, 8, shape, generator=g).float())


def _check(src, transpose, signs, random, device_src=None):
    from block_scaled_precision_amd import moe_mx as m
    x = src.cuda() if device_src is None else device_src
    codes, scales = m.mx4_quantize(x, transpose=transpose, signs=None if signs is None else signs.cuda(),
                                   random=None if random is None else random.cuda())
    oc, os_ = mx4.operand(src.double().numpy(), transpose, None if signs is None else signs.numpy(),
                          None if random is None else random.numpy())
    assert codes.shape == oc.shape and scales.shape == os_.shape
    bad = np.argwhere(scales.cpu().numpy() != os_)
    assert bad.size == 0, f"{len(bad)} scales differ, first at {bad[0]}"
    bad = np.argwhere(codes.cpu().numpy() != oc)
    assert bad.size == 0, f"{len(bad)} codes differ, first at {bad[0]}"
    return codes, scales


SHAPES = [(1, 1), (1, 32), (3, 33), (17, 128), (5, 200), (64, 512), (130, 257), (255, 64), (256, 65), (257, 130), (300, 1031),
          (1, 5000), (2000, 3), (2, 3, 5), (3, 100, 136), (7, 33, 64), (2, 300, 520)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("transpose,rotated,rounded", MODES)
def test_shapes(transpose, rotated, rounded, dtype):
    for shape in SHAPES:
        print_flush(f"mx4_quantize {shape} {dtype} transpose={transpose} signs={rotated} random={rounded}")
        x = _wide_range(shape, sum(shape)).to(dtype)
        _check(x, transpose, _signs(1) if rotated else None, gen.random_bytes(shape, 2, 82) if rounded else None)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rounded", [False, True])
def test_every_finite_bf16(transpose, rounded):
    """Every pattern next to a value 0 to 6 binades above the block's others; the largest, the
    subnormal and zeros of both signs among them."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF16)
    vals = bits[torch.isfinite(bits.float())]
    v = vals[:vals.numel() - vals.numel() % 31].reshape(-1, 31)
    for up in (0, 1, 3, 6):
        amax = v.float().abs().amax(1)
        ex = torch.frexp(torch.where(amax == 0, torch.ones_like(amax), amax)).exponent
        anchor = torch.ldexp(torch.ones_like(amax), (ex - 1 + up).clamp(max=127).float())
        anchor = torch.where(amax == 0, torch.ones_like(amax), anchor).to(BF16)
        x = torch.cat([v, anchor[:, None]], 1)
        x = x.T.contiguous() if transpose else x
        print_flush(f"mx4_quantize every bf16 up={up} transpose={transpose} random={rounded}")
        for dtype in (BF16, F32):
            _check(x.to(dtype), transpose, None, gen.random_bytes(x.shape, up, 83) if rounded else None)


@pytest.mark.parametrize("rounded", [False, True])
@pytest.mark.parametrize("transpose", [False, True])
def test_special_blocks(transpose, rounded):
    """Zeros and negative zeros, fp32 subnormals, the largest values, ties, each quarter and
    eighth between two codes."""
    g = torch.Generator().manual_seed(3)
    tiny = torch.randint(-(1 << 23) + 1, 1 << 23, (6, 32), generator=g).float() * 2.0 ** -149
    rows = [torch.zeros(32), torch.full((32,), -0.0), *tiny, torch.full((32,), torch.finfo(F32).max),
            torch.full((32,), -torch.finfo(F32).max), torch.full((32,), 2.0 ** -149), torch.full((32,), 2.0 ** -126),
            torch.arange(32) / 4, -torch.arange(32) / 4, torch.arange(32) / 8, torch.arange(32) / 5.25]
    x = torch.stack([r.float() for r in rows])
    x = torch.cat([x, x.flip(0)], 1)
    x = x.T.contiguous() if transpose else x
    for byte in (0, 1, 127, 128, 254, 255):
        random = torch.full(x.shape, byte, dtype=torch.uint8) if rounded else None
        _check(x, transpose, None, random)


@pytest.mark.parametrize("transpose", [False, True])
def test_rotation_in_fp32(transpose):
    """Every sum rounds (values of 24 bits in close binades); the rotated block overflows
    nothing that fits 2^122."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn((96, 160), generator=g) * torch.exp2(torch.randint(0, 20, (96, 160), generator=g).float())
    x[5] *= 2.0 ** 95
    x[:, 7] *= 2.0 ** -110
    for seed in range(4):
        _check(x, transpose, _signs(seed), None)
        _check(x, transpose, _signs(seed), gen.random_bytes(x.shape, seed, 84))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("transpose", [False, True])
def test_strides_and_given_outputs(dtype, transpose):
    """Rows at any distance and address of the type; what lies around is NaN, and outputs in
    the middle of guards."""
    from block_scaled_precision_amd import moe_mx as m
    for R, C, ld, at in ((40, 136, 136, 1), (130, 72, 77, 3), (300, 256, 264, 8), (33, 512, 520, 0)):
        print_flush(f"mx4_quantize strides {R}x{C} ld={ld} at={at}")
        x = _wide_range((R, C), R).to(dtype)
        buf = torch.full((at + R * ld + 8,), float("nan"), dtype=dtype, device="cuda")
        view = buf[at:at + R * ld].view(R, ld)[:, :C]
        view.copy_(x.cuda())
        want = _check(x, transpose, _signs(2), None, device_src=view)
        rows, K = want[0].shape[0], 2 * want[0].shape[1]
        codes = torch.full((3 * rows, K // 2), 99, dtype=torch.uint8, device="cuda")
        scales = torch.full((3 * rows, K // 32), 99, dtype=torch.uint8, device="cuda")
        m.mx4_quantize(view, transpose=transpose, signs=_signs(2).cuda(), codes=codes[rows:2 * rows],
                       scales=scales[rows:2 * rows])
        torch.cuda.synchronize()
        for t, w in ((codes, want[0]), (scales, want[1])):
            assert torch.equal(t[rows:2 * rows], w) and (t[:rows] == 99).all() and (t[2 * rows:] == 99).all()


def test_empty():
    from block_scaled_precision_amd import moe_mx as m
    for shape, transpose, want in (((0, 64), False, (0, 64)), ((0, 5, 7), True, (0, 7, 64)), ((0, 64), True, (64, 0))):
        codes, _ = m.mx4_quantize(torch.zeros(shape, device="cuda"), transpose=transpose)
        assert codes.shape == want, (shape, codes.shape)
    for transpose in (False, True):
        with pytest.raises(ValueError, match="at least one column"):
            m.mx4_quantize(torch.zeros((64, 0), device="cuda"), transpose=transpose)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_every_code_with_every_scale(dtype):
    """Exact but where bf16 or fp32 has no such value: past the largest one infinite (codes 4
    and 6 times 2^126 or 2^127), the NaN scale NaN; any row distance."""
    from block_scaled_precision_amd import moe_mx as m
    codes = torch.arange(256).to(torch.uint8).repeat(256).view(256, 256)
    scales = torch.arange(256).to(torch.uint8)[:, None].repeat(1, 16)
    want = mx4.values(codes.numpy(), scales.numpy())
    with np.errstate(over="ignore"):
        want = torch.from_numpy(want).to(F32).to(dtype)  # powers of two times 1, 1.5: no rounding
    for ld in (512, 519, 520):
        buf = torch.full((256, ld), 7.0, dtype=dtype, device="cuda")
        got = m.mx4_dequantize(codes.cuda(), scales.cuda(), dtype=dtype, out=buf[:, :512])
        assert torch.equal(torch.nan_to_num(got.cpu(), 5.0), torch.nan_to_num(want, 5.0))
        assert torch.equal(torch.isnan(got.cpu()), torch.isnan(want)) and (buf[:, 512:] == 7).all()
    assert torch.equal(torch.signbit(m.mx4_dequantize(codes.cuda(), scales.cuda(), dtype=dtype)[:255].cpu()),
                       torch.signbit(want[:255]))


def test_stochastic_rounding_keeps_the_mean():
    """256 equal rows with every byte once per column: the mean of the codes' values is within
    1/512 of the distance of the two neighbours (exact counts, no chance)."""
    from block_scaled_precision_amd import moe_mx as m
    row = gen.normal((1, 512), 5, 85)
    x = row.repeat(256, 1)
    random = ((torch.arange(256)[:, None] + 37 * torch.arange(512)[None]) % 256).to(torch.uint8)
    codes, scales = m.mx4_quantize(x.cuda(), random=random.cuda())
    v = m.mx4_dequantize(codes, scales, dtype=F32).double().cpu()
    gap = (v.amax(0) - v.amin(0))
    assert ((v.mean(0) - row[0].double()).abs() <= gap / 512 + (gap == 0) * 2.0 ** (scales[0].cpu().repeat_interleave(
        32).double() - 127) * 2 / 512).all()


def test_calls_at_once_and_captured():
    from block_scaled_precision_amd import moe_mx as m
    for kw in (dict(), dict(transpose=True), dict(signs=_signs(1).cuda()), dict(transpose=True, signs=_signs(1).cuda())):
        x = [gen.normal((700, 1000), 6 + i, 86).to(BF16).cuda() for i in range(2)]
        want = [m.mx4_quantize(t, **kw) for t in x]
        calls = [m.OpCall(m.mx4_quantize, t, **kw) for t in x]
        streams = [torch.cuda.Stream() for _ in x]
        torch.cuda.synchronize()
        for _ in range(20):
            for call, st in zip(calls, streams):
                with torch.cuda.stream(st):
                    call()
        torch.cuda.synchronize()
        for call, w in zip(calls, want):
            assert all(torch.equal(a, b) for a, b in zip(call(), w))
        graphs = []
        for call in calls:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = call()
                back = m.mx4_dequantize(*out)
            graphs.append((g, out, back))
        for i in (0, 1, 1, 0, 1):
            g, out, back = graphs[i]
            for t in (*out, back):
                t.zero_()
            g.replay()
            other = m.mx4_quantize(x[1 - i], **kw)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))
            assert all(torch.equal(a, b) for a, b in zip(other, want[1 - i]))
            assert torch.equal(back, m.mx4_dequantize(*want[i]))


@pytest.mark.parametrize("transpose", [False, True])
def test_offsets_past_32_bits(transpose):
    """More than 2^32 elements: the far corner against the same rows alone."""
    from block_scaled_precision_amd import moe_mx as m
    R, C = (1 << 20) + 512, 4096
    print_flush(f"mx4_quantize 64-bit offsets transpose={transpose}")
    x = torch.zeros((R, C), dtype=BF16, device="cuda")
    x[-512:] = gen.normal((512, C), 8, 87).to(BF16).cuda()
    codes, scales = m.mx4_quantize(x, transpose=transpose)
    c, s = m.mx4_quantize(x[-512:], transpose=transpose)
    if transpose:
        assert torch.equal(codes[:, -256:], c) and torch.equal(scales[:, -16:], s) and not codes[:, :-256].any()
        return
    assert torch.equal(codes[-512:], c) and torch.equal(scales[-512:], s) and not codes[:-512].any()
    back = m.mx4_dequantize(codes, scales)
    assert torch.equal(back[-512:], m.mx4_dequantize(c, s)) and not back[:-512].any()
