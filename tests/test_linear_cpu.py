"""Refusals of mx_linear, on the host: the C entry point with (never
dereferenced) addresses, and the binding with CPU tensors."""
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
PROBLEM = dict(M=4, N=64, K=128, groups=0, act=0, w_fmt=1, fn=0, bias_dtype=0, w_stride=0, w_scale_stride=0)
TENSORS = dict(a=A, w=A, w_scale=A, out=A)


def _call(p=(), t=(), ws=A, ws_bytes=1 << 60):
    _, L = _lib()
    p = m.MxLinearProblem(**{**PROBLEM, **dict(p)})
    t = m.MxLinearTensors(**{**TENSORS, **dict(t)})
    return L.mx_linear(ctypes.byref(p), ctypes.byref(t), ws, ws_bytes, None)


def _need(has_a_scale=False, **p):
    _, L = _lib()
    return L.mx_linear_workspace_bytes(ctypes.byref(m.MxLinearProblem(**{**PROBLEM, **p})), has_a_scale)


@host_only
@pytest.mark.parametrize("p,t,status", [
    ({}, {}, ARCH), (dict(M=0), dict(a=None, w=None, w_scale=None, out=None), OK),
    (dict(groups=3), dict(expert_offsets=A), ARCH), (dict(act=1), {}, ARCH), (dict(act=1), dict(a_scale=A), ARCH),
    (dict(w_fmt=2, fn=3, bias_dtype=1), dict(bias=A, mul=A, residual=A), ARCH),
    (dict(groups=2, w_stride=64 * 64 + 16, w_scale_stride=64 * 4 + 32), dict(expert_offsets=A), ARCH),
    (dict(M=-1), {}, INVALID), (dict(N=0), {}, INVALID), (dict(K=0), {}, INVALID), (dict(K=100), {}, INVALID),
    (dict(groups=-1), {}, INVALID), (dict(groups=1025), dict(expert_offsets=A), INVALID),
    (dict(act=2), {}, INVALID), (dict(w_fmt=0), {}, INVALID), (dict(fn=4), {}, INVALID), (dict(fn=-1), {}, INVALID),
    (dict(bias_dtype=2), {}, INVALID), (dict(w_stride=-16), {}, INVALID),
    (dict(groups=2, w_stride=64 * 64 - 16), dict(expert_offsets=A), INVALID),
    (dict(groups=2, w_stride=64 * 64 + 8), dict(expert_offsets=A), INVALID),
    (dict(groups=2, w_scale_stride=64 * 4 + 4), dict(expert_offsets=A), INVALID),
    (dict(groups=2), {}, INVALID), ({}, dict(expert_offsets=A), INVALID), ({}, dict(a_scale=A), INVALID),
    ({}, dict(a=None), INVALID), ({}, dict(w=None), INVALID), ({}, dict(w_scale=None), INVALID),
    ({}, dict(out=None), INVALID), ({}, dict(a=A + 2), INVALID), ({}, dict(w=A + 8), INVALID),
    ({}, dict(w_scale=A + 4), INVALID), ({}, dict(out=A + 2), INVALID), ({}, dict(mul=A + 2), INVALID),
    ({}, dict(residual=A + 8), INVALID), (dict(act=1), dict(a_scale=A + 1), INVALID),
    (dict(bias_dtype=1), dict(bias=A + 2), INVALID), (dict(bias_dtype=0), dict(bias=A + 2), ARCH),
    (dict(bias_dtype=0), dict(bias=A + 1), INVALID),
    (dict(N=60), {}, UNSUPPORTED), (dict(K=96), {}, UNSUPPORTED), (dict(w_fmt=3), {}, UNSUPPORTED),
    (dict(M=(1 << 30) + 1), {}, UNSUPPORTED), (dict(M=1 << 30, N=1 << 10), {}, UNSUPPORTED),
    (dict(K=1 << 24), {}, ARCH), (dict(K=(1 << 24) + 128), {}, UNSUPPORTED),
])
def test_c_abi_status(p, t, status):
    assert _call(p, t) == status


@host_only
def test_workspace():
    large = dict(M=4096, N=4096, K=1024, act=1)
    quant = 4096 * 1024 + 4096 * 32  # room for the quantized activations
    assert _need(**large) >= quant and _need(has_a_scale=True, **large) == 0 and _need(M=0, act=1) == 0
    assert _need() == 0 and _need(act=1) == 0  # few rows are quantized where they are read
    assert _need(groups=3) == 0 and _need(groups=3, **large) >= quant + _need(groups=3, has_a_scale=True, **large)
    assert _need(N=60, act=1) == 0
    p = dict(large, groups=3)
    need = _need(**p)
    for ws, n, status in ((A, need, ARCH), (A, need - 1, WORKSPACE), (None, need, WORKSPACE), (A + 128, need, INVALID)):
        assert _call(p, dict(expert_offsets=A), ws=ws, ws_bytes=n) == status


@host_only
@settings(**SETTINGS)
@given(M=SIZE, N=SIZE, K=SIZE, groups=SIZE, act=st.integers(-1, 2), fmt=st.integers(-1, 4), fn=st.integers(-1, 4),
       scaled=st.booleans())
def test_any_problem_gives_a_status(M, N, K, groups, act, fmt, fn, scaled):
    p = dict(M=M, N=N, K=K, groups=groups, act=act, w_fmt=fmt, fn=fn)
    need = _need(has_a_scale=scaled, **p)
    status = _call(p, dict(a_scale=A if scaled else None, expert_offsets=A if groups > 0 else None), ws_bytes=1 << 62)
    assert status in range(6) and need < 1 << 62


M_, N_, K_, G_ = 6, 16, 128, 3
U8, BF16, I32 = torch.uint8, torch.bfloat16, torch.int32


def _z(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


DENSE = dict(a=_z(M_, K_), w=_z(N_, K_ // 2, dtype=U8), w_scale=_z(N_, K_ // 32, dtype=U8), fmt="e2m1", act="bf16")
GROUPED = dict(DENSE, w=_z(G_, N_, K_ // 2, dtype=U8), w_scale=_z(G_, N_, K_ // 32, dtype=U8),
               expert_offsets=_z(G_ + 1, dtype=I32))


def test_valid_tensors_stop_at_the_device_check():
    both = _z(G_, 2 * N_, K_ // 2, dtype=U8)  # a gate half of a [gate; up] matrix
    for kw in (DENSE, GROUPED, dict(GROUPED, w=both[:, :N_]), dict(DENSE, bias=_z(N_, dtype=torch.float32)),
               dict(GROUPED, bias=_z(G_, N_), mul=_z(M_, N_), residual=_z(M_, N_), fn="gelu"),
               dict(DENSE, a=_z(M_, K_, dtype=U8), a_scale=_z(M_, K_ // 32, dtype=U8), act="mxfp8")):
        with pytest.raises(ValueError, match="GPU"):
            m.mx_linear(**kw)
        with pytest.raises(ValueError, match="GPU"):
            m.OpCall(m.mx_linear, **kw)


@pytest.mark.parametrize("base,change,msg", [
    (DENSE, dict(fmt="e4m3"), "weight format"), (DENSE, dict(act="fp16"), "activation precision"),
    (DENSE, dict(fn="swiglu"), "activation function"), (DENSE, dict(a=_z(K_)), "a: expected"),
    (DENSE, dict(a=_z(M_, K_, dtype=torch.float32)), "a: dtype"), (DENSE, dict(a=_z(K_, M_).t()), "multiple of 8|a: must be"),
    (DENSE, dict(a=_z(M_, 96)), "multiple of 8"), (DENSE, dict(w=GROUPED["w"]), "w: expected"),
    (GROUPED, dict(w=DENSE["w"]), "w: expected"), (DENSE, dict(w=_z(12, K_ // 2, dtype=U8)), "multiple of 8"),
    (DENSE, dict(w=_z(N_, K_, dtype=U8)), "w: shape"), (GROUPED, dict(w=_z(G_, N_, K_, dtype=U8)), "w: shape"),
    (GROUPED, dict(w=_z(G_, K_ // 2, N_, dtype=U8).transpose(1, 2)), "must be contiguous"),
    (GROUPED, dict(w=_z(1, N_, K_ // 2, dtype=U8).expand(G_, -1, -1)), "must not overlap"),
    (DENSE, dict(w_scale=_z(N_, 1, dtype=U8)), "w_scale: shape"), (GROUPED, dict(w_scale=_z(G_, N_, 4)), "w_scale: dtype"),
    (GROUPED, dict(expert_offsets=_z(G_, dtype=I32)), "expert_offsets: shape"),
    (GROUPED, dict(expert_offsets=_z(G_ + 1, dtype=torch.int64)), "expert_offsets: dtype"),
    (DENSE, dict(bias=_z(N_, dtype=torch.float16)), "bias: expected"), (DENSE, dict(bias=_z(N_ + 1)), "bias: shape"),
    (GROUPED, dict(bias=_z(N_)), "bias: shape"), (DENSE, dict(mul=_z(M_, N_, dtype=torch.float32)), "mul: dtype"),
    (DENSE, dict(residual=_z(M_ + 1, N_)), "residual: shape"), (DENSE, dict(a_scale=_z(M_, 4, dtype=U8)), "a_scale goes"),
    (DENSE, dict(a=_z(M_, K_, dtype=U8), a_scale=_z(M_, 3, dtype=U8), act="mxfp8"), "a_scale: shape"),
])
def test_refusals_of_the_binding(base, change, msg):
    with pytest.raises(ValueError, match=msg):
        m.mx_linear(**{**base, **change})
