"""ctypes binding of libmoe_mx.so (the C ABI declared in include/moe_mx.h).

Argument marshalling only: tensors are torch device tensors used as plain
device memory, streams are torch's current HIP stream, and every step of the
layer runs in the library's HIP kernels.  There is no fallback: if the library
is not built, or the device is not gfx950, calls raise.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_mx.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_ARCH, MOE_ERR_HIP = range(6)
MX_FORMATS = {"e2m1": 1, "e3m2": 2, "e4m3": 3}
FORMAT_BITS = {"e2m1": 4, "e3m2": 6, "e4m3": 8}
SRC_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
ACTS = {"bf16": 0, "mxfp8": 1}
LINEAR_FNS = {"none": 0, "silu": 1, "gelu": 2, "relu2": 3}
ACT_FNS = {"silu": 0, "relu2": 1, "swiglu_oai": 2}

# Every symbol include/moe_mx.h declares.
EXPORTS = ("mx_quantize", "moe_route_workspace_bytes", "moe_route", "moe_permute", "moe_permute_backward",
           "moe_unpermute", "moe_unpermute_backward", "moe_route_backward", "moe_balance_workspace_bytes", "moe_balance",
           "moe_balance_backward", "mx_gemm_workspace_bytes", "mx_gemm",
           "mx_linear_workspace_bytes", "mx_linear", "mx4_quantize", "mx4_dequantize", "mx4_linear_workspace_bytes",
           "mx4_linear",
           "moe_fused_workspace_bytes", "moe_fused", "moe_fused_workspace_offset", "moe_fused_noalloc",
           "moe_status_str", "moe_mx_version")
NOALLOC_SCRATCH_BYTES = 32 << 20  # MOE_NOALLOC_SCRATCH_BYTES


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_str(status)} (status {status})")


class MoeProblem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("w_fmt", ctypes.c_int),
                ("act", ctypes.c_int), ("I_shared", ctypes.c_int32), ("shared_weight", ctypes.c_float),
                ("local_expert_offset", ctypes.c_int32), ("local_num_experts", ctypes.c_int32),
                ("act_fn", ctypes.c_int), ("flags", ctypes.c_uint32)]


class MxLinearProblem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("groups", ctypes.c_int32),
                ("act", ctypes.c_int), ("w_fmt", ctypes.c_int), ("fn", ctypes.c_int), ("bias_dtype", ctypes.c_int),
                ("w_stride", ctypes.c_int64), ("w_scale_stride", ctypes.c_int64)]


class Mx4LinearProblem(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("groups", ctypes.c_int32),
                ("fn", ctypes.c_int), ("bias_dtype", ctypes.c_int), ("w_stride", ctypes.c_int64),
                ("w_scale_stride", ctypes.c_int64)]


class MxLinearTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "a", "a_scale", "w", "w_scale", "bias", "mul", "residual", "expert_offsets", "out")]


MOE_NUM_STAGES = 7
STAGES = ("route", "permute", "quant_x", "fc1", "fc2", "shared", "finalize")


class MoeTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "x", "router_logits", "topk_ids_in", "topk_w_in", "w1", "w1_scale", "w2", "w2_scale",
        "ws1", "ws1_scale", "ws2", "ws2_scale", "y", "topk_ids_out", "topk_w_out", "stage_events")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmoe_mx.so (built in-tree by block_scaled_precision_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m block_scaled_precision_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.mx_quantize.argtypes = [vp, ctypes.c_int, i64, i64, i64, ctypes.c_int, vp, vp, vp]
        L.mx_quantize.restype = ctypes.c_int
        L.moe_route_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_route_workspace_bytes.restype = sz
        L.moe_route.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_route.restype = ctypes.c_int
        L.moe_fused_workspace_bytes.argtypes = [ctypes.POINTER(MoeProblem)]
        L.moe_fused_workspace_bytes.restype = sz
        L.moe_fused.argtypes = [ctypes.POINTER(MoeProblem), ctypes.POINTER(MoeTensors), vp, sz, vp]
        L.moe_fused.restype = ctypes.c_int
        L.mx_gemm_workspace_bytes.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int]
        L.mx_gemm_workspace_bytes.restype = sz
        L.mx_gemm.argtypes = [vp, vp, i64, i64, i64, ctypes.c_int, vp, vp, ctypes.c_int, ctypes.c_float, vp, vp,
                              sz, vp]
        L.mx_gemm.restype = ctypes.c_int
        i = ctypes.c_int
        L.moe_permute.argtypes = [vp, i, i64, i32, i32, i32, i32, vp, vp, i32, i32, vp, i64, i32, vp, vp]
        L.moe_permute.restype = i
        L.moe_permute_backward.argtypes = [vp, i, i64, i32, vp, i32, i32, i32, vp, i64, vp]
        L.moe_permute_backward.restype = i
        L.moe_unpermute.argtypes = [vp, i, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, i64, vp]
        L.moe_unpermute.restype = i
        L.moe_unpermute_backward.argtypes = [vp, i, i64, vp, i64, i32, vp, vp, i32, i32, i32, vp, i64, vp, vp]
        L.moe_unpermute_backward.restype = i
        L.moe_route_backward.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
        L.moe_route_backward.restype = i
        L.moe_balance_workspace_bytes.argtypes = [i32, i32, i32]
        L.moe_balance_workspace_bytes.restype = sz
        L.moe_balance.argtypes = [vp, i64, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_balance.restype = i
        L.moe_balance_backward.argtypes = [vp, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, i64, vp]
        L.moe_balance_backward.restype = i
        L.mx_linear_workspace_bytes.argtypes = [ctypes.POINTER(MxLinearProblem), i]
        L.mx_linear_workspace_bytes.restype = sz
        L.mx_linear.argtypes = [ctypes.POINTER(MxLinearProblem), ctypes.POINTER(MxLinearTensors), vp, sz, vp]
        L.mx_linear.restype = i
        L.mx4_quantize.argtypes = [vp, i, i64, i64, i64, i64, i, vp, vp, vp, vp, vp]
        L.mx4_quantize.restype = i
        L.mx4_dequantize.argtypes = [vp, vp, i64, i64, vp, i, i64, vp]
        L.mx4_dequantize.restype = i
        L.mx4_linear_workspace_bytes.argtypes = [ctypes.POINTER(Mx4LinearProblem), i]
        L.mx4_linear_workspace_bytes.restype = sz
        L.mx4_linear.argtypes = [ctypes.POINTER(Mx4LinearProblem), ctypes.POINTER(MxLinearTensors), vp, sz, vp]
        L.mx4_linear.restype = i
        L.moe_fused_noalloc.argtypes = [ctypes.POINTER(MoeProblem), ctypes.POINTER(MoeTensors), vp]
        L.moe_fused_noalloc.restype = ctypes.c_int
        L.moe_fused_workspace_offset.argtypes = [ctypes.POINTER(MoeProblem), ctypes.c_int]
        L.moe_fused_workspace_offset.restype = sz
        L.moe_status_str.argtypes = [ctypes.c_int]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_mx_version.argtypes = []
        L.moe_mx_version.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _hold(stream, *tensors):
    """Keep the memory of tensors from reuse, once they are dropped, until `stream` has
    run what was launched on it.  True if that lasts: a record made under capture is
    for the capture's own allocations, and the graph's tensors have to outlive it."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return not torch.cuda.is_current_stream_capturing()


def _dev(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices ({dev} and {t.device})")


def _empty(shape, dtype, device, stream):
    """An output or workspace of a call on `stream`: from that stream's memory,
    and kept from reuse while the current stream may still read it."""
    if stream is None or stream == torch.cuda.current_stream(device):
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _require(t, name: str, dtype, shape):
    """The C ABI sees only a pointer: check what it will read or write."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _require_workspace(ws, need: int):
    if ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous():
        raise ValueError("workspace: expected a contiguous 1-D uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"workspace: {ws.numel()} bytes, need {need}")


# ------------------------------------------------------------ mx_quantize --

def mx_quantize(src: torch.Tensor, fmt: str, codes: torch.Tensor | None = None,
                scales: torch.Tensor | None = None, stream=None):
    """Block-quantize the last axis of a bf16/fp32 matrix [rows, cols] (or a
    batch [..., rows, cols], flattened) to MX codes + E8M0 scales."""
    if fmt not in MX_FORMATS:
        raise ValueError(f"unknown MX format {fmt!r}")
    if src.dtype not in SRC_DTYPES:
        raise ValueError(f"src: dtype {src.dtype}, expected bfloat16 or float32")
    if src.dim() < 1:
        raise ValueError("src: needs at least one axis")
    cols = src.shape[-1]
    if cols % 32 or cols == 0:
        raise ValueError(f"src: last axis {cols} is not a positive multiple of 32")
    rows = src.numel() // cols
    if src.is_contiguous():
        src2, ld = src.reshape(rows, cols), cols
    elif src.dim() == 2 and src.stride(-1) == 1 and src.stride(0) >= cols:
        src2, ld = src, src.stride(0)        # rows with a stride
    else:
        raise ValueError("src: must be contiguous, or 2-D with contiguous rows")
    nbytes = cols * FORMAT_BITS[fmt] // 8
    dev = src.device
    if codes is None:
        codes = _empty(src.shape[:-1] + (nbytes,), torch.uint8, dev, stream)
    if scales is None:
        scales = _empty(src.shape[:-1] + (cols // 32,), torch.uint8, dev, stream)
    _require(codes, "codes", torch.uint8, src.shape[:-1] + (nbytes,))
    _require(scales, "scales", torch.uint8, src.shape[:-1] + (cols // 32,))
    _dev(src, codes, scales)
    _check(lib().mx_quantize(_ptr(src2), SRC_DTYPES[src.dtype], rows, cols, ld, MX_FORMATS[fmt],
                             _ptr(codes), _ptr(scales), _stream(stream)), "mx_quantize")
    if stream is not None:
        _hold(stream, src, codes, scales)
    return codes, scales


# ---------------------------------------------------------------- route --

def moe_route_workspace_bytes(T: int, E: int, k: int) -> int:
    return lib().moe_route_workspace_bytes(T, E, k)


def moe_route(logits: torch.Tensor, k: int, workspace: torch.Tensor | None = None, stream=None):
    """-> (topk_ids [T,k] int32, topk_w [T,k] fp32, expert_offsets [E+1] int32,
    sorted_assign [T*k] int32)."""
    if logits.dim() != 2:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    _require(logits, "logits", torch.float32, (T, E))
    if not 1 <= k <= E:
        raise ValueError(f"k = {k} outside [1, E = {E}]")
    dev = logits.device
    ids = _empty((T, k), torch.int32, dev, stream)
    w = _empty((T, k), torch.float32, dev, stream)
    off = _empty((E + 1,), torch.int32, dev, stream)
    sa = _empty((T * k,), torch.int32, dev, stream)
    need = moe_route_workspace_bytes(T, E, k)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, dev, stream)
    _require_workspace(workspace, need)
    _dev(logits, workspace)
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _ptr(off), _ptr(sa),
                           _ptr(workspace), workspace.numel(), _stream(stream)), "moe_route")
    if stream is not None:
        _hold(stream, logits, ids, w, off, sa, workspace)
    return ids, w, off, sa


# ------------------------------------------------------- operator calls --
#
# The operators compute outside autograd.  Where gradients are on, they refuse a tensor
# that requires one.

class _Plan:
    """One checked and marshalled call of a C entry point: everything but the
    stream, which is its last argument."""
    __slots__ = ("name", "fn", "args", "result", "device", "keep", "recorded")

    def __init__(self, name, args, result, device, keep):
        # sizes cross the ABI as 32-bit integers, strides and addresses as 64-bit
        for v, ctype in zip(args, getattr(lib(), name).argtypes):
            if ctype is ctypes.c_int32 and not -2 ** 31 <= v < 2 ** 31:
                raise ValueError(f"{name}: size {v} does not fit 32 bits")
        self.name, self.fn, self.args = name, getattr(lib(), name), args
        self.result, self.device, self.keep = result, device, keep
        self.recorded = set()  # handles of the streams that the tensors' memory is kept for

    def launch(self, stream, prepared=False):
        """prepared: the plan may hold the last reference to its tensors, and their
        memory may come from another stream than the one it is launched on."""
        index = self.device.index
        if torch.cuda.current_device() != index:
            raise ValueError(f"{self.name}: tensors on {self.device}, which is not the current device")
        if stream is None:
            # the handle alone: torch.cuda.current_stream() makes an object for 2.6 of
            # the 6.9 us that a call of a small kernel costs the host
            handle = torch._C._cuda_getCurrentRawStream(index)
        elif stream.device == self.device:
            handle = stream.cuda_stream
        else:
            raise ValueError(f"{self.name}: stream on {stream.device}, tensors on {self.device}")
        status = self.fn(*self.args, handle)
        if status != MOE_OK:
            raise MoeError(status, self.name)
        if (prepared or stream is not None) and handle not in self.recorded:
            self._record(stream, handle)
        return self.result

    def _record(self, stream, handle):
        # once per stream is enough
        outputs = self.result if isinstance(self.result, tuple) else (self.result,)
        if _hold(torch.cuda.current_stream(self.device) if stream is None else stream, *outputs, *self.keep):
            self.recorded.add(handle)


_PLANNERS = {}  # operator -> function that plans a call of it


def _operator(planner):
    """The operator planned by `planner` (same arguments, and `stream`)."""
    def decorate(fn):
        _PLANNERS[fn] = planner
        return fn
    return decorate


class OpCall:
    """One operator call (moe_permute, moe_unpermute, moe_balance, their gradients,
    moe_route_backward, mx_linear, mx4_quantize, mx4_dequantize, mx4_linear) with its
    arguments checked and marshalled and its outputs allocated once, for loops that call it many times on the same
    buffers (their contents may change between calls): each call then costs the
    host only the C call.  The stream is the current one at each call unless
    one is given.  Calling returns the operator's outputs, the same tensors each
    time: its calls must not run at the same time (on two streams, or in two
    graphs), and it has to live as long as a graph that captured one.  It may be
    dropped, and so may its outputs and arguments, while a call is still running.

        combine = OpCall(moe_unpermute, rows, row_of, topk_w)
        y = combine()
    """

    def __init__(self, op, *args, stream=None, **kw):
        if op not in _PLANNERS:
            raise ValueError(f"{getattr(op, '__name__', op)!r} has no prepared form")
        self._plan = _PLANNERS[op](*args, stream=stream, **kw)
        self._stream = stream

    def __call__(self):
        return self._plan.launch(self._stream, prepared=True)


def _on_gpu(stream, *ts):
    """The one device of the given tensors, which has to be the current one
    (and the stream's)."""
    _dev(*ts)
    device = next(t.device for t in ts if t is not None)
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors on {device}, which is not the current device")
    if stream is not None and stream.device != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    return device


def _require_rows(t, name: str, dtype, shape) -> int:
    """A matrix with contiguous rows, any distance apart: its row stride."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    rows, cols = shape
    if rows <= 1:
        ld = cols
    else:
        ld = t.stride(0)
    if (cols > 1 and t.stride(1) != 1) or ld < cols:
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return ld


def _extent(t):
    """Address range of a tensor with nonnegative strides."""
    if t.numel() == 0:
        return 0, 0
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    start = t.data_ptr()
    return start, start + (last + 1) * t.element_size()


def _disjoint(outputs: dict, inputs: dict):
    """No output shares memory with an input or another output: refused from the first
    to the last element of each, so also between columns of one buffer."""
    ranges = [(n, _extent(t)) for n, t in inputs.items() if t is not None]
    for name, t in outputs.items():
        lo, hi = _extent(t)
        for other, (a, b) in ranges:
            if lo < b and a < hi:
                raise ValueError(f"{name} overlaps {other}")
        ranges.append((name, (lo, hi)))


def _no_graph(op: str, gradient: str, **tensors):
    """The operators record nothing for autograd: a tensor that waits for a gradient
    would silently get none."""
    if torch.is_grad_enabled():
        for name, t in tensors.items():
            if isinstance(t, torch.Tensor) and t.requires_grad:
                raise ValueError(f"{name} requires a gradient, which {op} does not record: call it under "
                                 f"torch.no_grad() or in a torch.autograd.Function ({gradient})")


# ------------------------------------------------------------- dispatch --

def _row_dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dtype not in SRC_DTYPES:
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16 or float32")
    if t.dim() != 2 or t.shape[1] == 0:
        raise ValueError(f"{name}: expected a matrix with at least one column")
    return t.dtype


def _tokens_slots(row_of):
    if not isinstance(row_of, torch.Tensor) or row_of.dim() != 2 or row_of.shape[1] == 0:
        raise ValueError("row_of: expected [T, k] with k >= 1")
    _require(row_of, "row_of", torch.int32, row_of.shape)
    return row_of.shape


def _plan_permute(x, sorted_assign, expert_offsets, k, local_offset=0, local_count=0, rows=None, row_of=None,
                  stream=None):
    _no_graph("moe_permute", "its gradient: moe_permute_backward", x=x, rows=rows)
    dtype = _row_dtype(x, "x")
    T, H = x.shape
    x_ld = _require_rows(x, "x", dtype, (T, H))
    if not isinstance(expert_offsets, torch.Tensor) or expert_offsets.dim() != 1 or expert_offsets.numel() < 2:
        raise ValueError("expert_offsets: expected [E + 1]")
    E = expert_offsets.numel() - 1
    if not 1 <= k <= E:
        raise ValueError(f"k = {k} outside [1, E = {E}]")
    if local_offset < 0 or local_count < 0 or local_offset + (local_count or E) > E:
        raise ValueError(f"local experts {local_offset} + {local_count or E} outside [0, E = {E}]")
    _require(expert_offsets, "expert_offsets", torch.int32, (E + 1,))
    _require(sorted_assign, "sorted_assign", torch.int32, (T * k,))
    device = _on_gpu(stream, x, sorted_assign, expert_offsets, rows, row_of)
    if rows is None:
        rows = _empty((T * min(k, local_count or E), H), dtype, device, stream)
    if row_of is None:
        row_of = _empty((T, k), torch.int32, device, stream)
    rows_ld = _require_rows(rows, "rows", dtype, (rows.shape[0], H))
    _require(row_of, "row_of", torch.int32, (T, k))
    _disjoint({"rows": rows, "row_of": row_of},
              {"x": x, "sorted_assign": sorted_assign, "expert_offsets": expert_offsets})
    return _Plan("moe_permute", (x.data_ptr(), SRC_DTYPES[dtype], x_ld, T, H, E, k, expert_offsets.data_ptr(),
                                 sorted_assign.data_ptr(), local_offset, local_count, rows.data_ptr(), rows_ld,
                                 rows.shape[0], row_of.data_ptr()),
                 (rows, row_of), device, (x, sorted_assign, expert_offsets))


@_operator(_plan_permute)
def moe_permute(x: torch.Tensor, sorted_assign: torch.Tensor, expert_offsets: torch.Tensor, k: int,
                local_offset: int = 0, local_count: int = 0, rows: torch.Tensor | None = None,
                row_of: torch.Tensor | None = None, stream=None):
    """Rows of x [T, H] (bf16 or fp32) sorted by expert -> (rows, row_of).

    sorted_assign [T*k] and expert_offsets [E+1] come from moe_route.  rows
    [>= T*min(k, local experts), H] holds the rows of the local experts
    [local_offset, + local_count) (0: all), the first of them at row 0; what lies
    behind the last local row is not written.  row_of [T, k] int32 is the row of
    each assignment, -1 where its expert is not local."""
    return _plan_permute(x, sorted_assign, expert_offsets, k, local_offset, local_count, rows, row_of,
                         stream).launch(stream)


def _plan_permute_backward(drows, row_of, dx=None, stream=None):
    _no_graph("moe_permute_backward", "of the second order", drows=drows, dx=dx)
    dtype = _row_dtype(drows, "drows")
    (R, H), (T, k) = drows.shape, _tokens_slots(row_of)
    ld = _require_rows(drows, "drows", dtype, (R, H))
    device = _on_gpu(stream, drows, row_of, dx)
    if dx is None:
        dx = _empty((T, H), dtype, device, stream)
    dx_ld = _require_rows(dx, "dx", dtype, (T, H))
    _disjoint({"dx": dx}, {"drows": drows, "row_of": row_of})
    return _Plan("moe_permute_backward", (drows.data_ptr(), SRC_DTYPES[dtype], ld, R, row_of.data_ptr(), T, H, k,
                                          dx.data_ptr(), dx_ld), dx, device, (drows, row_of))


@_operator(_plan_permute_backward)
def moe_permute_backward(drows: torch.Tensor, row_of: torch.Tensor, dx: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Gradient of moe_permute: dx [T, H], each token the sum (fp32, slot
    order) of its rows' gradients in drows [R, H]."""
    return _plan_permute_backward(drows, row_of, dx, stream).launch(stream)


def _plan_unpermute(rows, row_of, topk_w, residual=None, y=None, stream=None):
    _no_graph("moe_unpermute", "its gradient: moe_unpermute_backward", rows=rows, topk_w=topk_w, residual=residual, y=y)
    dtype = _row_dtype(rows, "rows")
    (R, H), (T, k) = rows.shape, _tokens_slots(row_of)
    ld = _require_rows(rows, "rows", dtype, (R, H))
    _require(topk_w, "topk_w", torch.float32, (T, k))
    res_ld = 0 if residual is None else _require_rows(residual, "residual", dtype, (T, H))
    device = _on_gpu(stream, rows, row_of, topk_w, residual, y)
    if y is None:
        y = _empty((T, H), dtype, device, stream)
    y_ld = _require_rows(y, "y", dtype, (T, H))
    in_place = residual is not None and residual.data_ptr() == y.data_ptr() and res_ld == y_ld
    _disjoint({"y": y}, {"rows": rows, "row_of": row_of, "topk_w": topk_w,
                         "residual": None if in_place else residual})
    return _Plan("moe_unpermute", (rows.data_ptr(), SRC_DTYPES[dtype], ld, R, row_of.data_ptr(), topk_w.data_ptr(),
                                   T, H, k, None if residual is None else residual.data_ptr(), res_ld, y.data_ptr(),
                                   y_ld), y, device, (rows, row_of, topk_w, residual))


@_operator(_plan_unpermute)
def moe_unpermute(rows: torch.Tensor, row_of: torch.Tensor, topk_w: torch.Tensor,
                  residual: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T, H] = residual + sum over slots of topk_w [T, k] * the slot's row of
    rows [R, H] (row_of [T, k] from moe_permute; absent rows are not read), in
    fp32 and rounded once.  y may be residual itself."""
    return _plan_unpermute(rows, row_of, topk_w, residual, y, stream).launch(stream)


def _plan_unpermute_backward(dy, rows, row_of, topk_w, drows=None, dw=None, stream=None):
    _no_graph("moe_unpermute_backward", "of the second order", dy=dy, rows=rows, topk_w=topk_w, drows=drows, dw=dw)
    dtype = _row_dtype(rows, "rows")
    (R, H), (T, k) = rows.shape, _tokens_slots(row_of)
    ld = _require_rows(rows, "rows", dtype, (R, H))
    dy_ld = _require_rows(dy, "dy", dtype, (T, H))
    _require(topk_w, "topk_w", torch.float32, (T, k))
    device = _on_gpu(stream, dy, rows, row_of, topk_w, drows, dw)
    if drows is None:
        drows = _empty((R, H), dtype, device, stream)
    if dw is None:
        dw = _empty((T, k), torch.float32, device, stream)
    drows_ld = _require_rows(drows, "drows", dtype, (R, H))
    _require(dw, "dw", torch.float32, (T, k))
    _disjoint({"drows": drows, "dw": dw}, {"dy": dy, "rows": rows, "row_of": row_of, "topk_w": topk_w})
    return _Plan("moe_unpermute_backward", (dy.data_ptr(), SRC_DTYPES[dtype], dy_ld, rows.data_ptr(), ld, R,
                                            row_of.data_ptr(), topk_w.data_ptr(), T, H, k, drows.data_ptr(),
                                            drows_ld, dw.data_ptr()),
                 (drows, dw), device, (dy, rows, row_of, topk_w))


@_operator(_plan_unpermute_backward)
def moe_unpermute_backward(dy: torch.Tensor, rows: torch.Tensor, row_of: torch.Tensor, topk_w: torch.Tensor,
                           drows: torch.Tensor | None = None, dw: torch.Tensor | None = None, stream=None):
    """Gradients of moe_unpermute -> (drows [R, H], dw [T, k] fp32): drows holds
    topk_w * dy in the rows that row_of names and leaves the others unwritten;
    dw is the dot product of dy and the row, 0 for an absent one.  The gradient
    of residual is dy."""
    return _plan_unpermute_backward(dy, rows, row_of, topk_w, drows, dw, stream).launch(stream)


def _plan_route_backward(topk_ids, topk_w, dw, num_experts, dlogits=None, stream=None):
    _no_graph("moe_route_backward", "of the second order", topk_w=topk_w, dw=dw, dlogits=dlogits)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2 or topk_ids.shape[1] == 0:
        raise ValueError("topk_ids: expected [T, k] with k >= 1")
    T, k = topk_ids.shape
    _require(topk_ids, "topk_ids", torch.int32, (T, k))
    _require(topk_w, "topk_w", torch.float32, (T, k))
    _require(dw, "dw", torch.float32, (T, k))
    if k > num_experts:
        raise ValueError(f"k = {k} outside [1, E = {num_experts}]")
    device = _on_gpu(stream, topk_ids, topk_w, dw, dlogits)
    if dlogits is None:
        dlogits = _empty((T, num_experts), torch.float32, device, stream)
    _require(dlogits, "dlogits", torch.float32, (T, num_experts))
    _disjoint({"dlogits": dlogits}, {"topk_ids": topk_ids, "topk_w": topk_w, "dw": dw})
    return _Plan("moe_route_backward", (topk_ids.data_ptr(), topk_w.data_ptr(), dw.data_ptr(), T, num_experts, k,
                                        dlogits.data_ptr()), dlogits, device, (topk_ids, topk_w, dw))


@_operator(_plan_route_backward)
def moe_route_backward(topk_ids: torch.Tensor, topk_w: torch.Tensor, dw: torch.Tensor, num_experts: int,
                       dlogits: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of moe_route's weights: dlogits [T, num_experts] fp32 from dw
    [T, k], zero for the experts a token did not choose."""
    return _plan_route_backward(topk_ids, topk_w, dw, num_experts, dlogits, stream).launch(stream)


# -------------------------------------------------------------- balance --

def _require_router(logits, k):
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2 or logits.shape[1] == 0:
        raise ValueError("logits: expected [T, E]")
    T, E = logits.shape
    ld = _require_rows(logits, "logits", torch.float32, (T, E))
    if not 1 <= k <= E:
        raise ValueError(f"k = {k} outside [1, E = {E}]")
    return T, E, ld


def _require_sequences(seq_offsets):
    """The number of sequences."""
    if seq_offsets is None:
        return 1
    if not isinstance(seq_offsets, torch.Tensor) or seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError("seq_offsets: expected [sequences + 1]")
    _require(seq_offsets, "seq_offsets", torch.int32, seq_offsets.shape)
    return seq_offsets.numel() - 1


def _data_ptr(t):
    return None if t is None else t.data_ptr()


def moe_balance_workspace_bytes(T: int, E: int, sequences: int = 1) -> int:
    return lib().moe_balance_workspace_bytes(T, E, sequences)


def _plan_balance(logits, topk_ids, mask=None, seq_offsets=None, loss=None, counts=None, tokens=None, lse=None,
                  workspace=None, stream=None):
    _no_graph("moe_balance", "its gradient: moe_balance_backward", logits=logits, loss=loss, lse=lse)
    if not isinstance(topk_ids, torch.Tensor) or topk_ids.dim() != 2:
        raise ValueError("topk_ids: expected [T, k]")
    k = topk_ids.shape[1]
    T, E, ld = _require_router(logits, k)
    _require(topk_ids, "topk_ids", torch.int32, (T, k))
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8):
            raise ValueError("mask: expected a bool or uint8 tensor")
        _require(mask, "mask", mask.dtype, (T,))
    S = _require_sequences(seq_offsets)
    for name, t, dtype, shape in (("loss", loss, torch.float32, (2,)), ("counts", counts, torch.int32, (S, E)),
                                  ("tokens", tokens, torch.int32, (S + 2,)), ("lse", lse, torch.float32, (T,))):
        if t is not None:
            _require(t, name, dtype, shape)
    device = _on_gpu(stream, logits, topk_ids, mask, seq_offsets, loss, counts, tokens, lse, workspace)
    if loss is None:
        loss = _empty((2,), torch.float32, device, stream)
    if counts is None:
        counts = _empty((S, E), torch.int32, device, stream)
    if tokens is None:
        tokens = _empty((S + 2,), torch.int32, device, stream)
    if lse is None:
        lse = _empty((T,), torch.float32, device, stream)
    need = moe_balance_workspace_bytes(T, E, S)
    if workspace is None and need:
        workspace = _empty((need,), torch.uint8, device, stream)
    outputs = {"loss": loss, "counts": counts, "tokens": tokens, "lse": lse}
    if workspace is not None:
        _require_workspace(workspace, need)
        outputs["workspace"] = workspace
    _disjoint(outputs, {"logits": logits, "topk_ids": topk_ids, "mask": mask, "seq_offsets": seq_offsets})
    return _Plan("moe_balance", (logits.data_ptr(), ld, topk_ids.data_ptr(), _data_ptr(mask), _data_ptr(seq_offsets),
                                 T, E, k, S, loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(), lse.data_ptr(),
                                 _data_ptr(workspace), 0 if workspace is None else workspace.numel()),
                 (loss, counts, tokens, lse), device, (logits, topk_ids, mask, seq_offsets, workspace))


@_operator(_plan_balance)
def moe_balance(logits: torch.Tensor, topk_ids: torch.Tensor, mask: torch.Tensor | None = None,
                seq_offsets: torch.Tensor | None = None, loss: torch.Tensor | None = None,
                counts: torch.Tensor | None = None, tokens: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """-> (loss [2] fp32: load balance and z-loss, counts [S, E] int32, tokens [S + 2]
    int32, lse [T] fp32) of router logits [T, E] fp32 and topk_ids [T, k] (moe_route).

    seq_offsets [S + 1] int32 are the sequences of a packed batch (None: one, of all
    tokens), mask [T] bool or uint8 the tokens that count; a token outside every
    sequence or with all logits -inf does not.  The balance loss is the mean over the
    sequences of E sum_e f_e P_e, f_e the share of assignments to expert e and P_e its mean
    probability; the z-loss the mean of lse^2.  tokens: each sequence's, all, and
    the number of sequences with one."""
    return _plan_balance(logits, topk_ids, mask, seq_offsets, loss, counts, tokens, lse, workspace,
                         stream).launch(stream)


def _plan_balance_backward(dloss, logits, counts, tokens, lse, k, seq_offsets=None, add=None, dlogits=None,
                           stream=None):
    _no_graph("moe_balance_backward", "of the second order", dloss=dloss, logits=logits, lse=lse, add=add,
              dlogits=dlogits)
    T, E, ld = _require_router(logits, k)
    S = _require_sequences(seq_offsets)
    _require(dloss, "dloss", torch.float32, (2,))
    _require(counts, "counts", torch.int32, (S, E))
    _require(tokens, "tokens", torch.int32, (S + 2,))
    _require(lse, "lse", torch.float32, (T,))
    add_ld = 0 if add is None else _require_rows(add, "add", torch.float32, (T, E))
    device = _on_gpu(stream, dloss, logits, counts, tokens, lse, seq_offsets, add, dlogits)
    if dlogits is None:
        dlogits = _empty((T, E), torch.float32, device, stream)
    out_ld = _require_rows(dlogits, "dlogits", torch.float32, (T, E))
    in_place = add is not None and add.data_ptr() == dlogits.data_ptr() and add_ld == out_ld
    _disjoint({"dlogits": dlogits}, {"dloss": dloss, "logits": logits, "counts": counts, "tokens": tokens, "lse": lse,
                                     "seq_offsets": seq_offsets, "add": None if in_place else add})
    return _Plan("moe_balance_backward", (dloss.data_ptr(), logits.data_ptr(), ld, counts.data_ptr(),
                                          tokens.data_ptr(), lse.data_ptr(), _data_ptr(seq_offsets), T, E, k, S,
                                          _data_ptr(add), add_ld, dlogits.data_ptr(), out_ld),
                 dlogits, device, (dloss, logits, counts, tokens, lse, seq_offsets, add))


@_operator(_plan_balance_backward)
def moe_balance_backward(dloss: torch.Tensor, logits: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor,
                         lse: torch.Tensor, k: int, seq_offsets: torch.Tensor | None = None,
                         add: torch.Tensor | None = None, dlogits: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Gradient of moe_balance's losses: dlogits [T, E] fp32 from dloss [2] fp32 and what
    moe_balance returned, plus add [T, E] (another gradient of the logits, such as
    moe_route_backward's; dlogits may be add itself).  The counts are constants; a token
    that does not count gets add, or 0."""
    return _plan_balance_backward(dloss, logits, counts, tokens, lse, k, seq_offsets, add, dlogits,
                                  stream).launch(stream)


# ---------------------------------------------------------------- gemm ---

def mx_gemm_workspace_bytes(M: int, N: int, K: int, act: str, w_fmt: str) -> int:
    return lib().mx_gemm_workspace_bytes(M, N, K, ACTS[act], MX_FORMATS[w_fmt])


def mx_gemm(a: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, fmt: str, act: str = "mxfp8",
            a_scale: torch.Tensor | None = None, alpha: float = 1.0, c: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """C [M, N] bf16 = alpha * A W^T over MX weights w [N, K*b/8] + w_scale
    [N, K/32].  a: [M, K] bf16 (act "bf16", or "mxfp8" quantized on the
    device), or E4M3 codes [M, K] uint8 with a_scale [M, K/32] (act "mxfp8")."""
    if fmt not in ("e2m1", "e3m2"):
        raise ValueError(f"weight format {fmt!r} is not e2m1 or e3m2")
    if act not in ACTS:
        raise ValueError(f"unknown activation precision {act!r}")
    if a.dim() != 2 or w.dim() != 2:
        raise ValueError("a and w must be 2-D")
    M, K = a.shape
    N = w.shape[0]
    b = FORMAT_BITS[fmt]
    if a_scale is None:
        _require(a, "a", torch.bfloat16, (M, K))
    else:
        if act != "mxfp8":
            raise ValueError("a_scale goes with act='mxfp8'")
        _require(a, "a", torch.uint8, (M, K))
        _require(a_scale, "a_scale", torch.uint8, (M, K // 32))
    _require(w, "w", torch.uint8, (N, K * b // 8))
    _require(w_scale, "w_scale", torch.uint8, (N, K // 32))
    if c is None:
        c = _empty((M, N), torch.bfloat16, a.device, stream)
    _require(c, "c", torch.bfloat16, (M, N))
    # MXFP8 from bf16: the quantized A; bf16 with few rows: the K split's partial sums
    need = mx_gemm_workspace_bytes(M, N, K, act, fmt) if a_scale is None else 0
    if workspace is None and need:
        workspace = _empty((need,), torch.uint8, a.device, stream)
    if workspace is not None:
        _require_workspace(workspace, need)
    _dev(a, a_scale, w, w_scale, c, workspace)
    _check(lib().mx_gemm(_ptr(a), _ptr(a_scale), M, N, K, ACTS[act], _ptr(w), _ptr(w_scale), MX_FORMATS[fmt],
                         alpha, _ptr(c), _ptr(workspace), 0 if workspace is None else workspace.numel(),
                         _stream(stream)), "mx_gemm")
    if stream is not None:
        _hold(stream, a, a_scale, w, w_scale, c, workspace)
    return c


# --------------------------------------------------------------- linear --

def _group_stride(t, name, shape, groups):
    """Bytes between the groups' matrices of t, each of them contiguous."""
    full = (groups, *shape) if groups else shape
    if groups == 0:
        _require(t, name, torch.uint8, full)
        return 0
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor")
    if t.dtype != torch.uint8:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {torch.uint8}")
    if tuple(t.shape) != full:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {full}")
    if not t[0].is_contiguous():
        raise ValueError(f"{name}: each group's matrix must be contiguous")
    if groups > 1 and (t.stride(0) < t[0].numel() or t.stride(0) % 16):
        raise ValueError(f"{name}: groups must not overlap and lie a multiple of 16 bytes apart")
    return t.stride(0) if groups > 1 else 0


def _call_linear(name, problem_of, a, a_bits, w, w_scale, fmt, a_scale, bias, fn, mul, residual, expert_offsets, out,
                 workspace, stream):
    """The checked call of entry point `name`: activations a [M, K] bf16, or with a_scale
    codes of a_bits bits; problem_of(M, N, K, groups, bias dtype, strides) -> its
    problem structure."""
    _no_graph(name, "of the user's own: there is no gradient through packed weights here", a=a, bias=bias, mul=mul,
              residual=residual, out=out)
    if fn not in LINEAR_FNS:
        raise ValueError(f"unknown activation function {fn!r}")
    grouped = expert_offsets is not None
    if not isinstance(a, torch.Tensor) or a.dim() != 2:
        raise ValueError("a: expected [M, K]")
    if not isinstance(w, torch.Tensor) or w.dim() != (3 if grouped else 2):
        raise ValueError("w: expected [groups, N, K*b/8] with expert_offsets, [N, K*b/8] without")
    M, K = a.shape
    if a_scale is not None:
        K = K * 8 // a_bits
    N, G = w.shape[-2], w.shape[0] if grouped else 0
    if N == 0 or N % 8 or K == 0 or K % 128:
        raise ValueError(f"N = {N} must be a positive multiple of 8, K = {K} of 128")
    if grouped and not 1 <= G <= 1024:
        raise ValueError(f"{G} groups outside [1, 1024]")
    if a_scale is None:
        _require(a, "a", torch.bfloat16, (M, K))
    else:
        _require(a, "a", torch.uint8, (M, K * a_bits // 8))
        _require(a_scale, "a_scale", torch.uint8, (M, K // 32))
    w_stride = _group_stride(w, "w", (N, K * FORMAT_BITS[fmt] // 8), G)
    s_stride = _group_stride(w_scale, "w_scale", (N, K // 32), G)
    if grouped:
        _require(expert_offsets, "expert_offsets", torch.int32, (G + 1,))
    if bias is not None:
        if not isinstance(bias, torch.Tensor) or bias.dtype not in SRC_DTYPES:
            raise ValueError("bias: expected a bfloat16 or float32 tensor")
        _require(bias, "bias", bias.dtype, (G, N) if grouped else (N,))
    for what, t in (("mul", mul), ("residual", residual)):
        if t is not None:
            _require(t, what, torch.bfloat16, (M, N))
    device = _on_gpu(stream, a, a_scale, w, w_scale, bias, mul, residual, expert_offsets, out, workspace)
    if out is None:
        out = _empty((M, N), torch.bfloat16, device, stream)
    _require(out, "out", torch.bfloat16, (M, N))
    problem = problem_of(M, N, K, G, 0 if bias is None else SRC_DTYPES[bias.dtype], w_stride, s_stride)
    need = getattr(lib(), name + "_workspace_bytes")(ctypes.byref(problem), a_scale is not None)
    if workspace is None and need:
        workspace = _empty((need,), torch.uint8, device, stream)
    if workspace is not None:
        _require_workspace(workspace, need)
    same = [t for t in (mul, residual) if t is not None and t.data_ptr() == out.data_ptr()]
    _disjoint({"out": out, **({} if workspace is None else {"workspace": workspace})},
              {"a": a, "a_scale": a_scale, "w": w, "w_scale": w_scale, "bias": bias, "expert_offsets": expert_offsets,
               "mul": None if any(t is mul for t in same) else mul,
               "residual": None if any(t is residual for t in same) else residual})
    if workspace is not None:
        _disjoint({"workspace": workspace}, {"mul": mul, "residual": residual})
    tensors = MxLinearTensors(*(None if t is None else t.data_ptr() for t in (
        a, a_scale, w, w_scale, bias, mul, residual, expert_offsets, out)))
    return _Plan(name, (ctypes.byref(problem), ctypes.byref(tensors),
                        None if workspace is None else workspace.data_ptr(),
                        0 if workspace is None else workspace.numel()),
                 out, device, (a, a_scale, w, w_scale, bias, mul, residual, expert_offsets, workspace))


def _plan_linear(a, w, w_scale, fmt, act="mxfp8", a_scale=None, bias=None, fn="none", mul=None, residual=None,
                 expert_offsets=None, out=None, workspace=None, stream=None):
    if fmt not in ("e2m1", "e3m2"):
        raise ValueError(f"weight format {fmt!r} is not e2m1 or e3m2")
    if act not in ACTS:
        raise ValueError(f"unknown activation precision {act!r}")
    if a_scale is not None and act != "mxfp8":
        raise ValueError("a_scale goes with act='mxfp8'")

    def problem(M, N, K, G, bias_dtype, w_stride, s_stride):
        return MxLinearProblem(M, N, K, G, ACTS[act], MX_FORMATS[fmt], LINEAR_FNS[fn], bias_dtype, w_stride, s_stride)
    return _call_linear("mx_linear", problem, a, 8, w, w_scale, fmt, a_scale, bias, fn, mul, residual, expert_offsets,
                        out, workspace, stream)


@_operator(_plan_linear)
def mx_linear(a: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, fmt: str, act: str = "mxfp8",
              a_scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, fn: str = "none",
              mul: torch.Tensor | None = None, residual: torch.Tensor | None = None,
              expert_offsets: torch.Tensor | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [M, N] bf16 = fn(A W^T + bias) * mul + residual, in fp32 and rounded once.

    a: [M, K] bf16 (act "bf16", or "mxfp8" quantized on the device), or E4M3
    codes [M, K] uint8 with a_scale [M, K/32].  w [N, K*b/8] + w_scale [N, K/32]
    packed MX weights; bias [N] bf16 or fp32; mul, residual [M, N] bf16 (out may
    be either); fn "none", "silu", "gelu" or "relu2".  With expert_offsets [G+1]
    int32 the rows of a are sorted by group (moe_permute) and w, w_scale and bias
    have a leading axis of G, one matrix per group; rows behind the last group
    are not written.  A shard of the experts passes its slice of moe_route's
    offsets."""
    return _plan_linear(a, w, w_scale, fmt, act, a_scale, bias, fn, mul, residual, expert_offsets, out, workspace,
                        stream).launch(stream)


# ------------------------------------------------------------------ mx4 --

def _plan_quantize4(src, transpose=False, signs=None, random=None, codes=None, scales=None, stream=None):
    _no_graph("mx4_quantize", "of the user's own: rounding has none", src=src)
    if not isinstance(src, torch.Tensor) or src.dim() not in (2, 3):
        raise ValueError("src: expected [rows, cols] or [batch, rows, cols]")
    if src.dtype not in SRC_DTYPES:
        raise ValueError(f"src: dtype {src.dtype}, expected bfloat16 or float32")
    rows, cols = src.shape[-2:]
    if cols == 0:
        raise ValueError("src: needs at least one column")
    if src.dim() == 2:
        batch, ld = 1, _require_rows(src, "src", src.dtype, (rows, cols))
    else:
        _require(src, "src", src.dtype, src.shape)
        batch, ld = src.shape[0], cols
    if signs is not None:
        _require(signs, "signs", torch.float32, (32,))
    if random is not None:
        _require(random, "random", torch.uint8, src.shape)
    out, K = (cols, rows) if transpose else (rows, cols)
    K = -(-K // 128) * 128
    device = _on_gpu(stream, src, signs, random, codes, scales)
    lead = src.shape[:-2]
    if codes is None:
        codes = _empty((*lead, out, K // 2), torch.uint8, device, stream)
    if scales is None:
        scales = _empty((*lead, out, K // 32), torch.uint8, device, stream)
    _require(codes, "codes", torch.uint8, (*lead, out, K // 2))
    _require(scales, "scales", torch.uint8, (*lead, out, K // 32))
    _disjoint({"codes": codes, "scales": scales}, {"src": src, "signs": signs, "random": random})
    return _Plan("mx4_quantize", (src.data_ptr(), SRC_DTYPES[src.dtype], batch, rows, cols, ld, int(bool(transpose)),
                                  _data_ptr(signs), _data_ptr(random), codes.data_ptr(), scales.data_ptr()),
                 (codes, scales), device, (src, signs, random))


@_operator(_plan_quantize4)
def mx4_quantize(src: torch.Tensor, transpose: bool = False, signs: torch.Tensor | None = None,
                 random: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
    """src [rows, cols] or [batch, rows, cols] (bf16 or fp32) as an operand of mx4_linear
    -> (codes [.., rows, K/2], scales [.., rows, K/32]) uint8, quantized to E2M1 along the
    columns, K their number rounded up to a multiple of 128 (zeros); with transpose,
    along the rows: (codes [.., cols, K/2], scales [.., cols, K/32]).

    signs [32] fp32 of +1 and -1 rotates every block of 32 by a Hadamard matrix (both
    operands of a product alike; a block whose sums leave fp32, which takes magnitudes of
    2^123 and more, gets the NaN scale); random, uint8 of src's shape, rounds stochastically and
    saturates nothing; without it the nearest code is taken, as mx_quantize does."""
    return _plan_quantize4(src, transpose, signs, random, codes, scales, stream).launch(stream)


def _plan_dequantize4(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    if not isinstance(codes, torch.Tensor) or codes.dim() < 2 or codes.dtype != torch.uint8:
        raise ValueError("codes: expected uint8 [.., rows, K/2]")
    lead, K = codes.shape[:-1], codes.shape[-1] * 2
    if K == 0 or K % 32:
        raise ValueError(f"codes: K = {K} is not a positive multiple of 32")
    if dtype not in SRC_DTYPES:
        raise ValueError(f"dtype {dtype}, expected bfloat16 or float32")
    _require(codes, "codes", torch.uint8, codes.shape)
    _require(scales, "scales", torch.uint8, (*lead, K // 32))
    _no_graph("mx4_dequantize", "of the user's own: codes have none", out=out)
    device = _on_gpu(stream, codes, scales, out)
    rows = codes.numel() // (K // 2)
    if out is None:
        out = _empty((*lead, K), dtype, device, stream)
    if codes.dim() == 2:
        ld = _require_rows(out, "out", dtype, (rows, K))
    else:
        _require(out, "out", dtype, (*lead, K))
        ld = K
    _disjoint({"out": out}, {"codes": codes, "scales": scales})
    return _Plan("mx4_dequantize", (codes.data_ptr(), scales.data_ptr(), rows, K, out.data_ptr(), SRC_DTYPES[dtype],
                                    ld), out, device, (codes, scales))


@_operator(_plan_dequantize4)
def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                   out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [.., rows, K] of E2M1 codes [.., rows, K/2] and scales [.., rows, K/32] as
    bf16 or fp32 (exact in both; 2^128 and more is infinite, scale code 255 NaN)."""
    return _plan_dequantize4(codes, scales, dtype, out, stream).launch(stream)


def _plan_linear4(a, w, w_scale, a_scale=None, bias=None, fn="none", mul=None, residual=None, expert_offsets=None,
                  out=None, workspace=None, stream=None):
    def problem(M, N, K, G, bias_dtype, w_stride, s_stride):
        return Mx4LinearProblem(M, N, K, G, LINEAR_FNS[fn], bias_dtype, w_stride, s_stride)
    return _call_linear("mx4_linear", problem, a, 4, w, w_scale, "e2m1", a_scale, bias, fn, mul, residual,
                        expert_offsets, out, workspace, stream)


@_operator(_plan_linear4)
def mx4_linear(a: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, a_scale: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, fn: str = "none", mul: torch.Tensor | None = None,
               residual: torch.Tensor | None = None, expert_offsets: torch.Tensor | None = None,
               out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """mx_linear with MXFP4 on both sides: out [M, N] bf16 = fn(A W^T + bias) * mul + residual.

    a: [M, K] bf16, quantized to E2M1 on the device, or E2M1 codes [M, K/2] uint8 with
    a_scale [M, K/32] (mx4_quantize).  w [N, K/2] + w_scale [N, K/32] E2M1 weights, with
    expert_offsets [G+1] one matrix per group; the other arguments are mx_linear's.
    Gradients of such a product are products of operands quantized transposed: dX of dY
    and W, dW of dY and X."""
    return _plan_linear4(a, w, w_scale, a_scale, bias, fn, mul, residual, expert_offsets, out, workspace,
                         stream).launch(stream)


# ---------------------------------------------------------------- fused --

@dataclass
class MoeWeights:
    """Packed MX weights of the local experts (canonical layout, device tensors)."""
    w1: torch.Tensor          # [L, 2I, H*b/8] uint8
    w1_scale: torch.Tensor    # [L, 2I, H/32] uint8
    w2: torch.Tensor          # [L, H, I*b/8] uint8
    w2_scale: torch.Tensor    # [L, H, I/32] uint8
    fmt: str                  # "e2m1" | "e3m2"
    ws1: torch.Tensor | None = None
    ws1_scale: torch.Tensor | None = None
    ws2: torch.Tensor | None = None
    ws2_scale: torch.Tensor | None = None


FLAG_FUSED_SMALL_BATCH = 1  # MOE_FLAG_FUSED_SMALL_BATCH


def make_problem(T, H, I, E, k, fmt, act, I_shared=0, shared_weight=1.0, local_offset=0, local_count=0,
                 act_fn="silu", fused_small_batch=False):
    return MoeProblem(T, H, I, E, k, MX_FORMATS[fmt], ACTS[act], I_shared, shared_weight,
                      local_offset, local_count, ACT_FNS[act_fn],
                      FLAG_FUSED_SMALL_BATCH if fused_small_batch else 0)


def moe_fused_workspace_bytes(problem: MoeProblem) -> int:
    return lib().moe_fused_workspace_bytes(ctypes.byref(problem))


WS_PARTS = {"expert_offsets": 0, "sorted_assign": 1, "h": 2, "h_scale": 3}


def moe_fused_workspace_offset(problem: MoeProblem, part: str):
    """Byte offset of an intermediate of moe_fused in its workspace, or None."""
    off = lib().moe_fused_workspace_offset(ctypes.byref(problem), WS_PARTS[part])
    return None if off == ctypes.c_size_t(-1).value else off


_FMT_NAMES = {v: k for k, v in MX_FORMATS.items()}


def check_fused_args(problem: MoeProblem, x, weights, router_logits=None, topk_ids_in=None,
                     topk_w_in=None, y=None, workspace=None, topk_ids_out=None, topk_w_out=None):
    """Every tensor of a moe_fused call against the problem: dtype, exact shape,
    contiguity, one GPU.  Raises ValueError before anything reaches the ABI."""
    p = problem
    T, H, I, E, k, Is = p.T, p.H, p.I, p.E, p.k, p.I_shared
    if p.w_fmt not in _FMT_NAMES or _FMT_NAMES[p.w_fmt] not in ("e2m1", "e3m2"):
        raise ValueError(f"problem: weight format code {p.w_fmt} is not e2m1 or e3m2")
    if weights.fmt != _FMT_NAMES[p.w_fmt]:
        raise ValueError(f"weights are {weights.fmt}, the problem says {_FMT_NAMES[p.w_fmt]}")
    if min(T, H, I, E, k, Is) < 0 or H == 0 or I == 0 or E == 0 or k == 0:
        raise ValueError("problem: negative or zero size")
    if H % 32 or I % 32 or Is % 32:
        raise ValueError("problem: H, I and I_shared must be multiples of 32")
    L = p.local_num_experts or E
    b = FORMAT_BITS[weights.fmt]
    _require(x, "x", torch.bfloat16, (T, H))
    _require(y, "y", torch.bfloat16, (T, H))
    if (topk_ids_in is None) != (topk_w_in is None):
        raise ValueError("topk_ids_in and topk_w_in go together")
    if topk_ids_in is None:
        if router_logits is None:
            raise ValueError("need router_logits or a precomputed top-k")
        _require(router_logits, "router_logits", torch.float32, (T, E))
    else:
        _require(topk_ids_in, "topk_ids_in", torch.int32, (T, k))
        _require(topk_w_in, "topk_w_in", torch.float32, (T, k))
        if router_logits is not None:
            _require(router_logits, "router_logits", torch.float32, (T, E))
    _require(weights.w1, "w1", torch.uint8, (L, 2 * I, H * b // 8))
    _require(weights.w1_scale, "w1_scale", torch.uint8, (L, 2 * I, H // 32))
    _require(weights.w2, "w2", torch.uint8, (L, H, I * b // 8))
    _require(weights.w2_scale, "w2_scale", torch.uint8, (L, H, I // 32))
    shared = (weights.ws1, weights.ws1_scale, weights.ws2, weights.ws2_scale)
    if Is > 0:
        _require(weights.ws1, "ws1", torch.uint8, (2 * Is, H * b // 8))
        _require(weights.ws1_scale, "ws1_scale", torch.uint8, (2 * Is, H // 32))
        _require(weights.ws2, "ws2", torch.uint8, (H, Is * b // 8))
        _require(weights.ws2_scale, "ws2_scale", torch.uint8, (H, Is // 32))
    else:
        shared = ()
    if topk_ids_out is not None:
        _require(topk_ids_out, "topk_ids_out", torch.int32, (T, k))
    if topk_w_out is not None:
        _require(topk_w_out, "topk_w_out", torch.float32, (T, k))
    if workspace is not None:
        _require_workspace(workspace, moe_fused_workspace_bytes(p))
    _dev(x, y, router_logits, topk_ids_in, topk_w_in, weights.w1, weights.w1_scale, weights.w2,
         weights.w2_scale, *shared, topk_ids_out, topk_w_out, workspace)


def moe_fused(problem: MoeProblem, x: torch.Tensor, weights: MoeWeights, router_logits=None,
              topk_ids_in=None, topk_w_in=None, y=None, workspace=None, topk_ids_out=None,
              topk_w_out=None, stream=None, stage_events=None):
    """Run the whole layer; returns y [T, H] bf16.

    stage_events: optional ctypes array of MOE_NUM_STAGES + 1 hipEvent_t
    handles (see HipEvents) recorded at the stage boundaries."""
    if y is None:
        y = _empty((problem.T, problem.H), torch.bfloat16, x.device, stream)
    need = moe_fused_workspace_bytes(problem)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, x.device, stream)
    check_fused_args(problem, x, weights, router_logits, topk_ids_in, topk_w_in, y, workspace,
                     topk_ids_out, topk_w_out)
    t = MoeTensors(*(None if v is None else v.data_ptr() for v in (
        x, router_logits, topk_ids_in, topk_w_in, weights.w1, weights.w1_scale, weights.w2,
        weights.w2_scale, weights.ws1, weights.ws1_scale, weights.ws2, weights.ws2_scale, y,
        topk_ids_out, topk_w_out)), None)
    if stage_events is not None:
        t.stage_events = ctypes.cast(stage_events, ctypes.c_void_p)
    _check(lib().moe_fused(ctypes.byref(problem), ctypes.byref(t), _ptr(workspace), workspace.numel(),
                           _stream(stream)), "moe_fused")
    if stream is not None:
        _hold(stream, *_fused_tensors(x, weights, router_logits, topk_ids_in, topk_w_in, y, workspace, topk_ids_out,
                                      topk_w_out))
    return y


def _fused_tensors(x, weights, *rest):
    return (x, weights.w1, weights.w1_scale, weights.w2, weights.w2_scale, weights.ws1, weights.ws1_scale, weights.ws2,
            weights.ws2_scale, *rest)


class FusedCall:
    """moe_fused with its arguments checked and marshalled once, for loops
    that call the layer many times on the same buffers (their contents may
    change between calls): each call then costs the host only the C call
    itself.  The stream is the current one at each call unless one is given.
    Calling returns y."""

    def __init__(self, problem: MoeProblem, x: torch.Tensor, weights: MoeWeights, router_logits=None,
                 topk_ids_in=None, topk_w_in=None, y=None, workspace=None, topk_ids_out=None,
                 topk_w_out=None, stream=None):
        if y is None:
            y = _empty((problem.T, problem.H), torch.bfloat16, x.device, stream)
        need = moe_fused_workspace_bytes(problem)
        if workspace is None:
            workspace = _empty((max(need, 1),), torch.uint8, x.device, stream)
        check_fused_args(problem, x, weights, router_logits, topk_ids_in, topk_w_in, y, workspace,
                         topk_ids_out, topk_w_out)
        self.y = y
        # the tensors stay referenced for as long as the call can run
        self._keep = (problem, x, weights, router_logits, topk_ids_in, topk_w_in, workspace, topk_ids_out,
                      topk_w_out)
        self._t = MoeTensors(*(None if v is None else v.data_ptr() for v in (
            x, router_logits, topk_ids_in, topk_w_in, weights.w1, weights.w1_scale, weights.w2,
            weights.w2_scale, weights.ws1, weights.ws1_scale, weights.ws2, weights.ws2_scale, y,
            topk_ids_out, topk_w_out)), None)
        self._p = ctypes.byref(problem)
        self._tp = ctypes.byref(self._t)
        self._ws = _ptr(workspace)
        self._wsn = workspace.numel()
        self._stream, self._handle = stream, None if stream is None else _stream(stream)
        self._tensors = _fused_tensors(x, weights, router_logits, topk_ids_in, topk_w_in, y, workspace, topk_ids_out,
                                       topk_w_out)
        self._recorded = set()  # handles of the streams that the tensors' memory is kept for
        self._fn = lib().moe_fused

    def __call__(self, stage_events=None):
        self._t.stage_events = None if stage_events is None else ctypes.cast(stage_events, ctypes.c_void_p)
        st = self._handle if self._handle is not None else _stream(None)
        status = self._fn(self._p, self._tp, self._ws, self._wsn, st)
        if status != MOE_OK:
            raise MoeError(status, "moe_fused")
        if st.value not in self._recorded:
            if _hold(torch.cuda.current_stream() if self._stream is None else self._stream, *self._tensors):
                self._recorded.add(st.value)
        return self.y


def moe_fused_noalloc(problem: MoeProblem, x: torch.Tensor, weights: MoeWeights, y: torch.Tensor,
                      router_logits=None, topk_ids_in=None, topk_w_in=None, topk_ids_out=None,
                      topk_w_out=None, stream=None):
    """The whole layer into the caller's y, with the library's static scratch
    as workspace: nothing is allocated (y must be given)."""
    if problem.T > 0:
        check_fused_args(problem, x, weights, router_logits, topk_ids_in, topk_w_in, y, None,
                         topk_ids_out, topk_w_out)
    t = MoeTensors(*(None if v is None else v.data_ptr() for v in (
        x, router_logits, topk_ids_in, topk_w_in, weights.w1, weights.w1_scale, weights.w2,
        weights.w2_scale, weights.ws1, weights.ws1_scale, weights.ws2, weights.ws2_scale, y,
        topk_ids_out, topk_w_out)), None)
    _check(lib().moe_fused_noalloc(ctypes.byref(problem), ctypes.byref(t), _stream(stream)), "moe_fused_noalloc")
    if stream is not None:
        _hold(stream, *_fused_tensors(x, weights, router_logits, topk_ids_in, topk_w_in, y, topk_ids_out, topk_w_out))
    return y


# ------------------------------------------------------------ HIP events --

class HipEvents:
    """A set of HIP events created with the HIP runtime that torch loaded (the
    library links the same one), for timing work on a given stream."""

    def __init__(self, n: int):
        self._hip = ctypes.CDLL("libamdhip64.so.7")
        self._hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                                   ctypes.c_void_p]
        self.handles = (ctypes.c_void_p * n)()
        for i in range(n):
            r = self._hip.hipEventCreate(ctypes.byref(self.handles, i * ctypes.sizeof(ctypes.c_void_p)))
            if r != 0:
                raise RuntimeError(f"hipEventCreate failed ({r})")

    def record(self, i: int, stream=None):
        r = self._hip.hipEventRecord(ctypes.c_void_p(self.handles[i]), _stream(stream))
        if r != 0:
            raise RuntimeError(f"hipEventRecord failed ({r})")

    def elapsed_ms(self, i: int, j: int) -> float:
        ms = ctypes.c_float()
        r = self._hip.hipEventElapsedTime(ctypes.byref(ms), ctypes.c_void_p(self.handles[i]),
                                          ctypes.c_void_p(self.handles[j]))
        if r != 0:
            raise RuntimeError(f"hipEventElapsedTime failed ({r})")
        return ms.value

    def __del__(self):
        try:
            for h in self.handles:
                if h:
                    self._hip.hipEventDestroy(ctypes.c_void_p(h))
        except Exception:
            pass
