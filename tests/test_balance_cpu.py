"""Refusals of moe_balance and its gradient, on the host: the C entry points with (never
dereferenced) addresses, and the binding with CPU tensors, where a call that passes every
check stops at the device check."""
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

CALLS = {
    "moe_balance": dict(logits=A, ld=8, ids=A, mask=A, offsets=A, T=4, E=8, k=2, S=3, loss=A, counts=A, tokens=A, lse=A,
                        ws=A, ws_bytes=1 << 60, stream=None),
    "moe_balance_backward": dict(dloss=A, logits=A, ld=8, counts=A, tokens=A, lse=A, offsets=A, T=4, E=8, k=2, S=3, add=A,
                                 add_ld=8, dlogits=A, dlogits_ld=8, stream=None),
}


def _call(name, **change):
    _, L = _lib()
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    return getattr(L, name)(*args.values())


@host_only
@pytest.mark.parametrize("name", sorted(CALLS))
def test_valid_calls_reach_the_architecture_check(name):
    assert _call(name) == ARCH and _call(name, offsets=None, S=1) == ARCH
    assert _call(name, E=1024, k=1024, ld=1024, **({} if name == "moe_balance" else dict(add_ld=1024, dlogits_ld=1024))) == ARCH
    if name == "moe_balance":
        assert _call(name, mask=None) == ARCH and _call(name, mask=A + 1) == ARCH
        assert _call(name, T=0, logits=None, ids=None, lse=None) == ARCH  # zeros are written
    else:
        assert _call(name, add=None, add_ld=0) == ARCH
        assert _call(name, T=0, logits=None, lse=None, dlogits=None) == OK


@host_only
@pytest.mark.parametrize("name,change,status", [
    (n, c, s) for n in sorted(CALLS) for c, s in [
        (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025, ld=1025), INVALID), (dict(k=0), INVALID),
        (dict(k=9), INVALID), (dict(S=0), INVALID), (dict(S=-1), INVALID), (dict(offsets=None), INVALID),
        (dict(T=1 << 30), UNSUPPORTED), (dict(S=1 << 28), UNSUPPORTED), (dict(S=(1 << 20) + 1), UNSUPPORTED),
        (dict(ld=7), INVALID), (dict(add_ld=7), INVALID),
        (dict(dlogits_ld=7), INVALID), (dict(dlogits_ld=-8), INVALID),
        *((dict([(p, None)]), INVALID) for p in ("logits", "ids", "loss", "counts", "tokens", "lse", "dloss", "dlogits")),
        *((dict([(p, A + 2)]), INVALID) for p in ("logits", "ids", "offsets", "loss", "counts", "tokens", "lse", "dloss",
                                                  "add", "dlogits")),
    ] if set(c) <= set(CALLS[n])])
def test_refusals_of_the_c_abi(name, change, status):
    assert _call(name, **change) == status


@host_only
def test_workspace():
    _, L = _lib()
    need = L.moe_balance_workspace_bytes
    assert need(64, 384, 1) == 0 and need(4, 8, 3) == 0  # a few tokens need none
    big = need(10000, 384, 3)
    assert big > 0 and need(20000, 384, 3) >= big and need(10000, 384, 30) > big and need(-1, 8, 1) == need(1, 0, 1) == 0
    for ws, n, status in ((A, big, ARCH), (A, big - 1, WORKSPACE), (None, big, WORKSPACE), (A + 64, big, INVALID)):
        assert _call("moe_balance", T=10000, E=384, ld=384, ws=ws, ws_bytes=n) == status
    assert _call("moe_balance", ws=None, ws_bytes=0) == ARCH


@host_only
@settings(**SETTINGS)
@given(T=SIZE, E=SIZE, k=SIZE, S=SIZE, ld=SIZE)
def test_any_sizes_give_a_status(T, E, k, S, ld):
    values = dict(T=T, E=E, k=k, S=S, ld=ld, add_ld=ld, dlogits_ld=ld)
    for name, args in CALLS.items():
        assert _call(name, **{x: v for x, v in values.items() if x in args}) in range(6)


def _z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


T, E, K, S = 6, 8, 2, 3
I32 = torch.int32
BINDING = {
    m.moe_balance: dict(logits=_z(T, E), topk_ids=_z(T, K, dtype=I32)),
    m.moe_balance_backward: dict(dloss=_z(2), logits=_z(T, E), counts=_z(1, E, dtype=I32), tokens=_z(3, dtype=I32),
                                 lse=_z(T), k=K),
}
SEQS = dict(seq_offsets=_z(S + 1, dtype=I32))


@pytest.mark.parametrize("op", list(BINDING), ids=lambda f: f.__name__)
def test_valid_tensors_stop_at_the_device_check(op):
    more = dict(SEQS) if op is m.moe_balance else dict(SEQS, counts=_z(S, E, dtype=I32), tokens=_z(S + 2, dtype=I32))
    for kw in (BINDING[op], {**BINDING[op], **more}):
        with pytest.raises(ValueError, match="GPU"):
            op(**kw)
        with pytest.raises(ValueError, match="GPU"):
            m.OpCall(op, **kw)
    wide = _z(T, 2 * E)
    with pytest.raises(ValueError, match="GPU"):
        op(**{**BINDING[op], "logits": wide[:, :E]})
    for mask in (_z(T, dtype=torch.bool), _z(T, dtype=torch.uint8)):
        with pytest.raises(ValueError, match="GPU"):
            m.moe_balance(**BINDING[m.moe_balance], mask=mask)


@pytest.mark.parametrize("op,change,msg", [
    (m.moe_balance, dict(logits=_z(T, E, dtype=torch.bfloat16)), "logits: dtype"),
    (m.moe_balance, dict(logits=_z(T)), "logits: expected"), (m.moe_balance, dict(logits=_z(T, 0)), "logits: expected"),
    (m.moe_balance, dict(logits=_z(E, T).t()), "rows must be contiguous"),
    (m.moe_balance, dict(topk_ids=_z(T, K)), "topk_ids: dtype"),
    (m.moe_balance, dict(topk_ids=_z(T, E + 1, dtype=I32)), "outside"),
    (m.moe_balance, dict(topk_ids=_z(T, 0, dtype=I32)), "outside"),
    (m.moe_balance, dict(topk_ids=_z(T + 1, K, dtype=I32)), "topk_ids: shape"),
    (m.moe_balance, dict(mask=_z(T)), "mask: expected"), (m.moe_balance, dict(mask=_z(T + 1, dtype=torch.bool)), "mask: shape"),
    (m.moe_balance, dict(seq_offsets=_z(1, dtype=I32)), "seq_offsets: expected"),
    (m.moe_balance, dict(seq_offsets=_z(3)), "seq_offsets: dtype"),
    (m.moe_balance, dict(loss=_z(1)), "loss: shape"), (m.moe_balance, dict(counts=_z(2, E, dtype=I32)), "counts: shape"),
    (m.moe_balance, dict(tokens=_z(2, dtype=I32)), "tokens: shape"), (m.moe_balance, dict(lse=_z(T - 1)), "lse: shape"),
    (m.moe_balance_backward, dict(dloss=_z(1)), "dloss: shape"),
    (m.moe_balance_backward, dict(counts=_z(1, E)), "counts: dtype"),
    (m.moe_balance_backward, dict(SEQS), "counts: shape"),
    (m.moe_balance_backward, dict(SEQS, counts=_z(S, E, dtype=I32)), "tokens: shape"),
    (m.moe_balance_backward, dict(k=0), "outside"), (m.moe_balance_backward, dict(k=E + 1), "outside"),
    (m.moe_balance_backward, dict(add=_z(T, E + 1)), "add: shape"),
    (m.moe_balance_backward, dict(add=_z(1, E).expand(T, E)), "must not overlap"),
    (m.moe_balance_backward, dict(lse=_z(T, dtype=torch.float64)), "lse: dtype"),
])
def test_refusals_of_the_binding(op, change, msg):
    with pytest.raises(ValueError, match=msg):
        op(**{**BINDING[op], **change})


@pytest.mark.parametrize("op,name", [(m.moe_balance, "logits"), (m.moe_balance, "loss"), (m.moe_balance, "lse"),
                                     *((m.moe_balance_backward, n) for n in ("dloss", "logits", "lse", "add", "dlogits"))])
def test_a_tensor_that_requires_a_gradient_is_refused(op, name):
    shapes = dict(logits=(T, E), loss=(2,), lse=(T,), dloss=(2,), add=(T, E), dlogits=(T, E))
    kw = {**BINDING[op], name: _z(*shapes[name]).requires_grad_()}
    with pytest.raises(ValueError, match=f"^{name} requires a gradient, which {op.__name__} does not"):
        op(**kw)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        op(**kw)
