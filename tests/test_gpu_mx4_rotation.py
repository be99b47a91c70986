"""mx4_quantize's rotation at the end of fp32's range: magnitudes below 2^123 add up inside it; a
block whose sums overflow has the NaN scale, and no other block changes."""
import numpy as np
import pytest
import torch

from oracle import mx4
from tests.conftest import has_gpu
from tests.helpers import print_flush

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not has_gpu(), reason="needs a GPU")]

F32, BF16 = torch.float32, torch.bfloat16


def _blocks(dtype, seed):
    """Rows of four blocks: around 2^122, at the largest magnitude below 2^123 (all of one sign
    after the signs, so that one sum holds all 32), past it, and single huge values."""
    g = torch.Generator().manual_seed(seed)
    signs = torch.where(torch.rand(32, generator=g) < 0.5, -1.0, 1.0)
    most = torch.tensor(2.0).pow(123).to(dtype)
    bits = most.view(torch.int16 if dtype == BF16 else torch.int32)
    below = (bits - 1).view(dtype).float()
    huge = torch.finfo(dtype).max
    normal = torch.randn((40, 128), generator=g)
    rows = [normal[0] * 2.0 ** 120, torch.cat([signs] * 4) * below, torch.cat([-signs] * 4) * below,
            torch.where(torch.rand(128, generator=g) < 0.5, -below, below)]
    for i in range(12):  # one block overflows or comes close, the others are ordinary
        r = normal[4 + i].clone()
        r[32 * (i % 4):32 * (i % 4) + 32] *= 2.0 ** (122 + i % 6 * 0.8)
        rows.append(r)
    for i in range(8):  # one or two of the largest values, alone or among zeros
        r = normal[20 + i] * (i % 2)
        r[(37 * i) % 128] = huge
        if i > 3:
            r[(37 * i + 5) % 128] = -huge
        rows.append(r)
    return torch.stack(rows).clamp(-huge, huge).to(dtype), signs


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rounded", [False, True])
def test_rotation_up_to_the_end_of_fp32(transpose, rounded, dtype):
    from block_scaled_precision_amd import moe_mx as m
    print_flush(f"mx4_quantize rotation transpose={transpose} random={rounded} {dtype}")
    for seed in range(4):
        x, signs = _blocks(dtype, seed)
        random = torch.randint(0, 256, x.shape, dtype=torch.uint8) if rounded else None
        if transpose:
            x, random = x.T.contiguous(), None if random is None else random.T.contiguous()
        codes, scales = m.mx4_quantize(x.cuda(), transpose=transpose, signs=signs.cuda(),
                                       random=None if random is None else random.cuda())
        oc, os_ = mx4.operand(x.double().numpy(), transpose, signs.numpy(), None if random is None else random.numpy())
        assert np.array_equal(scales.cpu().numpy(), os_)
        assert (os_[:4] < 255).all() and (os_ == 255).sum() >= 4  # both kinds are there
        fine = np.repeat(os_ < 255, 16, axis=-1)
        assert np.array_equal(codes.cpu().numpy()[fine], oc[fine])
        values = m.mx4_dequantize(codes, scales, dtype=F32).cpu()
        assert np.array_equal(torch.isnan(values).numpy(), np.repeat(os_ == 255, 32, axis=-1))
