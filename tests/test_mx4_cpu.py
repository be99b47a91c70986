"""Refusals of mx4_quantize, mx4_dequantize and mx4_linear, on the host: the C entry points
with (never dereferenced) addresses, and the binding with CPU tensors."""
import ctypes

import pytest
import torch
from hypothesis import given, settings
from hypothesis import strategies as st

from block_scaled_precision_amd import moe_mx as m
from tests.conftest import has_gpu
from tests.test_abi_cpu import _lib
from tests.test_abi_fuzz_cpu import SETTINGS, SIZE

host_only = pytest.mark.skipif(has_gpu(), reason="host-only checks with fake device pointers")
A = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE, ARCH = 0, 1, 2, 3, 4
QUANT = dict(src=A, dtype=0, batch=2, rows=6, cols=40, ld=40, transpose=0, signs=A, random=A, codes=A, scales=A, stream=None)
VALUES = dict(codes=A, scales=A, rows=6, cols=64, dst=A, dtype=0, ld=64, stream=None)
PROBLEM = dict(M=4, N=64, K=128, groups=0, fn=0, bias_dtype=0, w_stride=0, w_scale_stride=0)
TENSORS = dict(a=A, w=A, w_scale=A, out=A)


def _call(name, base, **change):
    _, L = _lib()
    assert set(change) <= set(base)
    return getattr(L, name)(*{**base, **change}.values())


@host_only
@pytest.mark.parametrize("change,status", [
    ({}, ARCH), (dict(transpose=1), ARCH), (dict(signs=None, random=None), ARCH), (dict(dtype=1, ld=41), ARCH),
    (dict(src=A + 2, random=A + 1), ARCH), (dict(cols=1, ld=1), ARCH),
    (dict(rows=0, src=None, codes=None, scales=None), OK), (dict(batch=0, src=None), OK),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(batch=-1), INVALID), (dict(ld=39), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID), (dict(transpose=2), INVALID), (dict(transpose=-1), INVALID),
    (dict(src=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(src=A + 1), INVALID),
    (dict(dtype=1, src=A + 2), INVALID), (dict(codes=A + 8), INVALID), (dict(scales=A + 2), INVALID),
    (dict(signs=A + 2), INVALID), (dict(rows=(1 << 30) + 1), UNSUPPORTED), (dict(cols=(1 << 30) + 1, ld=1 << 31), UNSUPPORTED),
    (dict(rows=1 << 30, cols=1 << 20, ld=1 << 20), UNSUPPORTED), (dict(batch=1 << 30, rows=1 << 20, transpose=1), UNSUPPORTED),
])
def test_quantize_status(change, status):
    assert _call("mx4_quantize", QUANT, **change) == status


@host_only
@pytest.mark.parametrize("change,status", [
    ({}, ARCH), (dict(dtype=1, ld=65), ARCH), (dict(rows=0, codes=None, scales=None, dst=None), OK),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=48), INVALID), (dict(ld=63), INVALID),
    (dict(dtype=2), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dst=None), INVALID),
    (dict(codes=A + 2), INVALID), (dict(dst=A + 1), INVALID), (dict(dtype=1, dst=A + 2), INVALID),
    (dict(rows=(1 << 30) + 1), UNSUPPORTED),
])
def test_dequantize_status(change, status):
    assert _call("mx4_dequantize", VALUES, **change) == status


def _linear(p=(), t=(), ws=A, ws_bytes=1 << 60):
    _, L = _lib()
    p = m.Mx4LinearProblem(**{**PROBLEM, **dict(p)})
    t = m.MxLinearTensors(**{**TENSORS, **dict(t)})
    return L.mx4_linear(ctypes.byref(p), ctypes.byref(t), ws, ws_bytes, None)


def _need(has_a_scale=False, **p):
    _, L = _lib()
    return L.mx4_linear_workspace_bytes(ctypes.byref(m.Mx4LinearProblem(**{**PROBLEM, **p})), has_a_scale)


@host_only
@pytest.mark.parametrize("p,t,status", [
    ({}, {}, ARCH), ({}, dict(a_scale=A), ARCH), (dict(M=0), dict(a=None, w=None, w_scale=None, out=None), OK),
    (dict(groups=3), dict(expert_offsets=A), ARCH), (dict(fn=3, bias_dtype=1), dict(bias=A, mul=A, residual=A), ARCH),
    (dict(groups=2, w_stride=64 * 64 + 16, w_scale_stride=64 * 4 + 32), dict(expert_offsets=A), ARCH),
    (dict(M=-1), {}, INVALID), (dict(N=0), {}, INVALID), (dict(K=0), {}, INVALID), (dict(K=100), {}, INVALID),
    (dict(groups=-1), {}, INVALID), (dict(groups=1025), dict(expert_offsets=A), INVALID), (dict(fn=4), {}, INVALID),
    (dict(fn=-1), {}, INVALID), (dict(bias_dtype=2), {}, INVALID), (dict(w_stride=-16), {}, INVALID),
    (dict(groups=2, w_stride=64 * 64 - 16), dict(expert_offsets=A), INVALID),
    (dict(groups=2, w_scale_stride=64 * 4 + 4), dict(expert_offsets=A), INVALID),
    (dict(groups=2), {}, INVALID), ({}, dict(expert_offsets=A), INVALID), ({}, dict(a=None), INVALID),
    ({}, dict(w=None), INVALID), ({}, dict(w_scale=None), INVALID), ({}, dict(out=None), INVALID),
    ({}, dict(a=A + 2), INVALID), ({}, dict(a_scale=A + 4), INVALID), ({}, dict(w=A + 8), INVALID),
    ({}, dict(mul=A + 2), INVALID), ({}, dict(residual=A + 8), INVALID), (dict(bias_dtype=1), dict(bias=A + 2), INVALID),
    (dict(N=60), {}, UNSUPPORTED), (dict(K=96), {}, UNSUPPORTED), (dict(M=(1 << 30) + 1), {}, UNSUPPORTED),
    (dict(M=1 << 30, N=1 << 10), {}, UNSUPPORTED), (dict(K=1 << 24), {}, ARCH), (dict(K=(1 << 24) + 128), {}, UNSUPPORTED),
])
def test_linear_status(p, t, status):
    assert _linear(p, t) == status


@host_only
def test_linear_workspace():
    large = dict(M=4096, N=4096, K=1024)
    quant = 4096 * 1024 // 2 + 4096 * 32  # room for the quantized activations
    assert _need(**large) >= quant and _need(has_a_scale=True, **large) == 0 and _need(M=0) == 0
    assert _need() == 0  # few rows are quantized where they are read
    assert _need(N=60) == 0 and _need(groups=3, **large) >= quant + _need(groups=3, has_a_scale=True, **large)
    p = dict(large, groups=3)
    need = _need(**p)
    for ws, n, status in ((A, need, ARCH), (A, need - 1, WORKSPACE), (None, need, WORKSPACE), (A + 128, need, INVALID)):
        assert _linear(p, dict(expert_offsets=A), ws=ws, ws_bytes=n) == status


@host_only
@settings(**SETTINGS)
@given(M=SIZE, N=SIZE, K=SIZE, groups=SIZE, fn=st.integers(-1, 4), scaled=st.booleans(), dtype=st.integers(-1, 2),
       transpose=st.integers(-1, 2), ld=SIZE)
def test_any_problem_gives_a_status(M, N, K, groups, fn, scaled, dtype, transpose, ld):
    p = dict(M=M, N=N, K=K, groups=groups, fn=fn)
    need = _need(has_a_scale=scaled, **p)
    status = _linear(p, dict(a_scale=A if scaled else None, expert_offsets=A if groups > 0 else None), ws_bytes=1 << 62)
    assert status in range(6) and need < 1 << 62
    assert _call("mx4_quantize", QUANT, dtype=dtype, batch=groups, rows=M, cols=N, ld=ld, transpose=transpose) in range(6)
    assert _call("mx4_dequantize", VALUES, dtype=dtype, rows=M, cols=K, ld=ld) in range(6)


M_, N_, K_, G_ = 6, 16, 128, 3
U8, BF16, I32 = torch.uint8, torch.bfloat16, torch.int32


def _z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


DENSE = dict(a=_z(M_, K_), w=_z(N_, K_ // 2, dtype=U8), w_scale=_z(N_, K_ // 32, dtype=U8))
CODES = dict(DENSE, a=_z(M_, K_ // 2, dtype=U8), a_scale=_z(M_, K_ // 32, dtype=U8))
GROUPED = dict(DENSE, w=_z(G_, N_, K_ // 2, dtype=U8), w_scale=_z(G_, N_, K_ // 32, dtype=U8),
               expert_offsets=_z(G_ + 1, dtype=I32))
VALID = {
    m.mx4_linear: [DENSE, CODES, GROUPED, dict(GROUPED, bias=_z(G_, N_), mul=_z(M_, N_), residual=_z(M_, N_), fn="gelu")],
    m.mx4_quantize: [dict(src=_z(5, 7)), dict(src=_z(2, 5, 7, dtype=torch.float32), transpose=True),
                     dict(src=_z(5, 14)[:, :7], signs=_z(32, dtype=torch.float32), random=_z(5, 7, dtype=U8)),
                     dict(src=_z(5, 7), codes=_z(5, 64, dtype=U8), scales=_z(5, 4, dtype=U8))],
    m.mx4_dequantize: [dict(codes=_z(5, 32, dtype=U8), scales=_z(5, 2, dtype=U8)),
                       dict(codes=_z(2, 5, 32, dtype=U8), scales=_z(2, 5, 2, dtype=U8), dtype=torch.float32)],
}


@pytest.mark.parametrize("op", list(VALID), ids=lambda f: f.__name__)
def test_valid_tensors_stop_at_the_device_check(op):
    for kw in VALID[op]:
        with pytest.raises(ValueError, match="GPU"):
            op(**kw)
        with pytest.raises(ValueError, match="GPU"):
            m.OpCall(op, **kw)


@pytest.mark.parametrize("base,change,msg", [
    (DENSE, dict(a=_z(M_, K_ // 2, dtype=U8)), "multiple of 8|dtype"), (CODES, dict(a=_z(M_, K_, dtype=U8)), "a_scale: shape"),
    (CODES, dict(a=_z(M_, K_ // 2)), "a: dtype"), (CODES, dict(a_scale=_z(M_, 3, dtype=U8)), "a_scale: shape"),
    (DENSE, dict(a=_z(K_)), "a: expected"), (DENSE, dict(a=_z(M_, 96)), "multiple of 8"),
    (DENSE, dict(w=GROUPED["w"]), "w: expected"), (GROUPED, dict(w=DENSE["w"]), "w: expected"),
    (DENSE, dict(w=_z(N_, K_, dtype=U8)), "w: shape"), (DENSE, dict(fn="swiglu"), "activation function"),
    (DENSE, dict(bias=_z(N_, dtype=torch.float16)), "bias: expected"), (DENSE, dict(mul=_z(M_, N_ + 8)), "mul: shape"),
    (DENSE, dict(residual=_z(M_, N_, dtype=torch.float32)), "residual: dtype"),
    (GROUPED, dict(expert_offsets=_z(G_, dtype=I32)), "expert_offsets: shape"),
    (DENSE, dict(out=_z(M_, N_, dtype=torch.float32)), "GPU|out: dtype"),
])
def test_refusals_of_linear(base, change, msg):
    with pytest.raises(ValueError, match=msg):
        m.mx4_linear(**{**base, **change})


@pytest.mark.parametrize("op,kw,msg", [
    (m.mx4_quantize, dict(src=_z(5)), "src: expected"), (m.mx4_quantize, dict(src=_z(2, 2, 2, 2)), "src: expected"),
    (m.mx4_quantize, dict(src=_z(5, 7, dtype=torch.float16)), "src: dtype"), (m.mx4_quantize, dict(src=_z(5, 0)), "column"),
    (m.mx4_quantize, dict(src=_z(7, 5).t()), "rows must be contiguous"),
    (m.mx4_quantize, dict(src=_z(2, 5, 14)[:, :, :7]), "src: must be contiguous"),
    (m.mx4_quantize, dict(src=_z(5, 7), signs=_z(16, dtype=torch.float32)), "signs: shape"),
    (m.mx4_quantize, dict(src=_z(5, 7), signs=_z(32)), "signs: dtype"),
    (m.mx4_quantize, dict(src=_z(5, 7), random=_z(7, 5, dtype=U8)), "random: shape"),
    (m.mx4_quantize, dict(src=_z(5, 7), random=_z(5, 7, dtype=torch.int8)), "random: dtype"),
    (m.mx4_dequantize, dict(codes=_z(5, 32), scales=_z(5, 2, dtype=U8)), "codes: expected"),
    (m.mx4_dequantize, dict(codes=_z(32, dtype=U8), scales=_z(2, dtype=U8)), "codes: expected"),
    (m.mx4_dequantize, dict(codes=_z(5, 24, dtype=U8), scales=_z(5, 1, dtype=U8)), "multiple of 32"),
    (m.mx4_dequantize, dict(codes=_z(5, 32, dtype=U8), scales=_z(5, 1, dtype=U8)), "scales: shape"),
    (m.mx4_dequantize, dict(codes=_z(5, 32, dtype=U8), scales=_z(5, 2, dtype=U8), dtype=torch.float16), "dtype"),
])
def test_refusals_of_the_operands(op, kw, msg):
    with pytest.raises(ValueError, match=msg):
        op(**kw)


@pytest.mark.parametrize("op,kw,name", [
    (m.mx4_linear, DENSE, "a"), (m.mx4_linear, dict(DENSE, bias=_z(N_)), "bias"),
    (m.mx4_linear, dict(DENSE, mul=_z(M_, N_)), "mul"), (m.mx4_linear, dict(DENSE, residual=_z(M_, N_)), "residual"),
    (m.mx4_quantize, dict(src=_z(5, 7)), "src"),
])
def test_a_tensor_that_requires_a_gradient_is_refused(op, kw, name):
    kw = {**kw, name: kw[name].clone().requires_grad_()}
    with pytest.raises(ValueError, match=f"^{name} requires a gradient, which {op.__name__} does not"):
        op(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        op(**kw)
