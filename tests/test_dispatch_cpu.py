"""Refusals of the dispatch operators, on the host: the C entry points with
(never dereferenced) addresses, and the binding with CPU tensors, where a call
that passes every check stops at the device check."""
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
OK, INVALID, UNSUPPORTED, ARCH = 0, 1, 2, 4

# valid calls, argument by argument
CALLS = {
    "moe_permute": dict(x=A, dtype=0, x_ld=64, T=4, H=64, E=8, k=2, offsets=A, order=A, lo=0, n=0, rows=A, rows_ld=64,
                        num_rows=8, row_of=A, stream=None),
    "moe_permute_backward": dict(drows=A, dtype=0, drows_ld=64, num_rows=8, row_of=A, T=4, H=64, k=2, dx=A, dx_ld=64,
                                 stream=None),
    "moe_unpermute": dict(rows=A, dtype=0, rows_ld=64, num_rows=8, row_of=A, w=A, T=4, H=64, k=2, residual=A,
                          residual_ld=64, y=A, y_ld=64, stream=None),
    "moe_unpermute_backward": dict(dy=A, dtype=0, dy_ld=64, rows=A, rows_ld=64, num_rows=8, row_of=A, w=A, T=4, H=64,
                                   k=2, drows=A, drows_ld=64, dw=A, stream=None),
    "moe_route_backward": dict(ids=A, w=A, dw=A, T=4, E=8, k=2, dlogits=A, stream=None),
}


def _call(name, **change):
    _, L = _lib()
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    return getattr(L, name)(*args.values())


@host_only
@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_call_reaches_the_architecture_check(name):
    assert _call(name) == ARCH
    assert _call(name, T=0) == OK
    if "num_rows" in CALLS[name]:
        matrices = {n: None for n in ("rows", "drows") if n in CALLS[name]}
        assert _call(name, num_rows=0, **matrices) == ARCH  # no rows: their matrices are not needed
        assert _call(name, **{next(iter(matrices)): None}) == INVALID
    if name == "moe_unpermute":
        assert _call(name, residual=None) == ARCH


@host_only
@pytest.mark.parametrize("name,change,status", [
    (n, c, s) for n in sorted(CALLS) for c, s in [
        (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(H=0), INVALID), (dict(H=(1 << 24) + 1), UNSUPPORTED),
        (dict(T=1 << 30, k=2), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(dtype=-1), INVALID),
        (dict(num_rows=-1), INVALID), (dict(row_of=None), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID),
        (dict(x=None), INVALID), (dict(dx=None), INVALID), (dict(y=None), INVALID), (dict(dy=None), INVALID),
        (dict(offsets=None), INVALID), (dict(order=None), INVALID), (dict(ids=None), INVALID),
        (dict(dlogits=None), INVALID), (dict(x_ld=63), INVALID), (dict(rows_ld=63), INVALID),
        (dict(dy_ld=0), INVALID), (dict(y_ld=-64), INVALID), (dict(dx_ld=1), INVALID), (dict(drows_ld=63), INVALID),
        (dict(residual_ld=63), INVALID), (dict(x=A + 1), INVALID), (dict(y=A + 1), INVALID), (dict(dy=A + 1), INVALID),
        (dict(rows=A + 1), INVALID), (dict(drows=A + 1), INVALID), (dict(residual=A + 1), INVALID),
        (dict(E=1025), INVALID), (dict(E=0), INVALID), (dict(k=9, E=8), INVALID), (dict(lo=-1), INVALID),
        (dict(lo=4, n=5), INVALID), (dict(n=-1), INVALID), (dict(lo=1, n=0), INVALID),
    ] if set(c) <= set(CALLS[n])])
def test_refusals_of_the_c_abi(name, change, status):
    if name == "moe_route_backward" and change == dict(T=1 << 30, k=2):
        status = UNSUPPORTED
    assert _call(name, **change) == status


@host_only
@settings(**SETTINGS)
@given(T=SIZE, H=SIZE, E=SIZE, k=SIZE, lo=SIZE, n=SIZE, R=SIZE, ld=SIZE, dtype=st.integers(-1, 2))
def test_any_sizes_give_a_status(T, H, E, k, lo, n, R, ld, dtype):
    values = dict(T=T, H=H, E=E, k=k, lo=lo, n=n, num_rows=R, dtype=dtype, x_ld=ld, rows_ld=ld, drows_ld=ld, dx_ld=ld,
                  y_ld=ld, dy_ld=ld, residual_ld=ld)
    for name, args in CALLS.items():
        assert _call(name, **{x: v for x, v in values.items() if x in args}) in range(6)


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


T, H, E, K = 6, 40, 8, 2
I32, BF16 = torch.int32, torch.bfloat16
BINDING = {
    m.moe_permute: dict(x=_z(T, H), sorted_assign=_z(T * K, dtype=I32), expert_offsets=_z(E + 1, dtype=I32), k=K),
    m.moe_permute_backward: dict(drows=_z(9, H), row_of=_z(T, K, dtype=I32)),
    m.moe_unpermute: dict(rows=_z(9, H), row_of=_z(T, K, dtype=I32), topk_w=_z(T, K)),
    m.moe_unpermute_backward: dict(dy=_z(T, H), rows=_z(9, H), row_of=_z(T, K, dtype=I32), topk_w=_z(T, K)),
    m.moe_route_backward: dict(topk_ids=_z(T, K, dtype=I32), topk_w=_z(T, K), dw=_z(T, K), num_experts=E),
}


@pytest.mark.parametrize("op", list(BINDING), ids=lambda f: f.__name__)
def test_valid_tensors_stop_at_the_device_check(op):
    with pytest.raises(ValueError, match="GPU"):
        op(**BINDING[op])
    with pytest.raises(ValueError, match="GPU"):
        m.OpCall(op, **BINDING[op])


@pytest.mark.parametrize("op,change,msg", [
    (m.moe_permute, dict(x=_z(T, H, dtype=torch.float16)), "x: dtype"),
    (m.moe_permute, dict(x=_z(T)), "x: expected a matrix"),
    (m.moe_permute, dict(x=_z(H, T).t()), "rows must be contiguous"),
    (m.moe_permute, dict(x=_z(1, H).expand(T, H)), "must not overlap"),
    (m.moe_permute, dict(x=_z(T, 0)), "at least one column"),
    (m.moe_permute, dict(k=E + 1), "outside"),
    (m.moe_permute, dict(k=0), "outside"),
    (m.moe_permute, dict(local_offset=5, local_count=4), "local experts"),
    (m.moe_permute, dict(local_offset=1), "local experts"),
    (m.moe_permute, dict(local_offset=-1, local_count=1), "local experts"),
    (m.moe_permute, dict(sorted_assign=_z(T * K - 1, dtype=I32)), "sorted_assign: shape"),
    (m.moe_permute, dict(sorted_assign=_z(T * K, dtype=torch.int64)), "sorted_assign: dtype"),
    (m.moe_permute, dict(expert_offsets=_z(E + 1)), "expert_offsets: dtype"),
    (m.moe_permute, dict(expert_offsets=_z(1, dtype=I32)), "expert_offsets: expected"),
    (m.moe_permute_backward, dict(row_of=_z(T, K)), "row_of: dtype"),
    (m.moe_permute_backward, dict(row_of=_z(T, 0, dtype=I32)), "row_of: expected"),
    (m.moe_permute_backward, dict(row_of=_z(K, T, dtype=I32).t()), "row_of: must be contiguous"),
    (m.moe_unpermute, dict(topk_w=_z(T, K, dtype=BF16)), "topk_w: dtype"),
    (m.moe_unpermute, dict(topk_w=_z(T, K + 1)), "topk_w: shape"),
    (m.moe_unpermute, dict(residual=_z(T, H, dtype=BF16)), "residual: dtype"),
    (m.moe_unpermute, dict(residual=_z(T + 1, H)), "residual: shape"),
    (m.moe_unpermute_backward, dict(dy=_z(T, H + 1)), "dy: shape"),
    (m.moe_unpermute_backward, dict(rows=_z(9, H, dtype=BF16)), "dy: dtype"),
    (m.moe_route_backward, dict(num_experts=1), "outside"),
    (m.moe_route_backward, dict(dw=_z(T, K, dtype=BF16)), "dw: dtype"),
    (m.moe_route_backward, dict(topk_ids=_z(T, K, dtype=torch.int64)), "topk_ids: dtype"),
    (m.moe_route_backward, dict(topk_ids=_z(T, 0, dtype=I32)), "topk_ids: expected"),
])
def test_refusals_of_the_binding(op, change, msg):
    with pytest.raises(ValueError, match=msg):
        op(**{**BINDING[op], **change})


def test_prepared_form_of_other_functions_is_refused():
    with pytest.raises(ValueError, match="no prepared form"):
        m.OpCall(m.moe_route, _z(T, E), K)


def test_overlap_and_size_checks():
    base = _z(T, 2 * H)
    with pytest.raises(ValueError, match="y overlaps rows"):
        m._disjoint({"y": base[:, :H]}, {"rows": base[:, H:]})
    m._disjoint({"y": base[:3]}, {"rows": base[3:], "w": None})
    with pytest.raises(ValueError, match="b overlaps a"):
        m._disjoint({"a": base[:3], "b": base[2:4]}, {})
    assert ctypes.c_int32(1 << 31).value < 0  # what an unchecked size would turn into
    with pytest.raises(ValueError, match="32 bits"):
        m._Plan("moe_route_backward", (A, A, A, 1 << 31, 8, 2, A), None, None, ())
