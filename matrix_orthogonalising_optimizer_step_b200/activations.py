"""Activation operators around the optimizer step (see the last section of
include/muonclip.h): activations in 8 bits, the root-mean-square norm with the
residual's addition, weight gradients from 8-bit inputs, and tokens sorted by
expert and back.

They make what the step takes: the layer inputs x of ``qk_max_logit`` and
``mla_max_logit`` (which accept an ``Act8``) and the gradients of ``muon_step``.
Results are allocated with torch on the stream that the call runs on unless
``out`` is given; so is scratch, unless ``workspace`` is.  All calls can be
captured into a CUDA graph.

No call records an autograd graph: results never require gradients, whatever
the inputs do.  Backward passes are calls of their own, made by the training loop or
from the ``backward`` of a ``torch.autograd.Function``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import (MC_ACT_E4M3, MC_ACT_INT8, MC_BF16, MC_F32, McAct8, _check, _need_cuda_contig, _one_device, _ptr,
               load_library)

ACT_BLOCK = 32
_CODE = {torch.float32: MC_F32, torch.bfloat16: MC_BF16}
_FMT = {"e4m3": MC_ACT_E4M3, "int8": MC_ACT_INT8}


class Act8(NamedTuple):
    """An activation in 8 bits: ``q`` uint8 [rows, >= cols] codes, ``scale`` uint8
    [rows, >= ceil(cols / 32)] scale bytes (rows of both whole 16 bytes), ``shape``
    the logical shape (rows = product of all but the last) and ``fmt`` "e4m3" or
    "int8".  A value is code * 2^(scale - 127); scale 255 marks a block of NaN."""
    q: "torch.Tensor"
    scale: "torch.Tensor"
    shape: tuple
    fmt: str


class RmsNorm(NamedTuple):
    """h (x itself without a residual), y (bf16 tensor or Act8) and rstd (fp32 [rows])."""
    h: "torch.Tensor"
    y: object
    rstd: "torch.Tensor"


class ExpertPlan(NamedTuple):
    """The order that ``expert_sort`` gives: ``offsets`` int32 [E + 1], ``source``
    int32 [T * K] (pair t * K + k of each sorted row, -1 behind the last) and
    ``position`` int32 [T, K] (row of each pair, -1 if dropped)."""
    offsets: "torch.Tensor"
    source: "torch.Tensor"
    position: "torch.Tensor"


# The current stream's handle and the current device, without a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _enter(device, stream):
    """Makes the device (and the stream, if one is given) current; returns what
    has to be left again, or None where nothing had to be done."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        cm = torch.cuda.stream(stream)
    elif device.index == _current_device():
        return None
    else:
        cm = torch.cuda.device(device)
    cm.__enter__()
    return cm


def _one_dev(first, *others):
    """The device of ``first``; raises unless every other (non-None) tensor is on it."""
    at = first.get_device()
    for t in others:
        if t is not None and t.get_device() != at:
            _one_device([first, *others])
    return first.device


def _dtype_code(t):
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _rows_cols(shape):
    if len(shape) == 2:
        return shape[0], shape[1]
    rows = 1
    for n in shape[:-1]:
        rows *= int(n)
    return rows, int(shape[-1])


def _need_matrix(t, name):
    if not (t.is_cuda and t.is_contiguous()):
        _need_cuda_contig(t, name)
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name} must have at least one column, got shape {tuple(t.shape)}")


def _need_like(t, name, other, other_name):
    _need_cuda_contig(t, name)
    if t.shape != other.shape or t.dtype != other.dtype:
        raise ValueError(f"{name} must have {other_name}'s shape and type")


def _fmt_code(fmt):
    code = _FMT.get(fmt)
    if code is None:
        raise ValueError(f"fmt must be 'e4m3' or 'int8', got {fmt!r}")
    return code


def _act8_struct(a, name):
    q, s, shape, fmt = a
    code = _fmt_code(fmt)
    u8 = torch.uint8
    if not (q.is_cuda and s.is_cuda):
        raise ValueError(f"{name}.q and {name}.scale must be CUDA tensors")
    if not (q.dtype is u8 and s.dtype is u8):
        raise TypeError(f"{name}.q and {name}.scale must be uint8")
    qs, ss = q.shape, s.shape
    if not (len(qs) == 2 and len(ss) == 2 and q.is_contiguous() and s.is_contiguous()):
        raise ValueError(f"{name}.q and {name}.scale must be contiguous 2D tensors")
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name}.shape must have at least one column, got {tuple(shape)}")
    rows, cols = _rows_cols(shape)
    if qs[0] != rows or ss[0] != rows:
        raise ValueError(f"{name}: q and scale must have {rows} rows, got {qs[0]} and {ss[0]}")
    if qs[1] < cols or qs[1] % 16 or ss[1] * ACT_BLOCK < cols or ss[1] % 16:
        raise ValueError(f"{name}: rows of q and scale must be whole 16 bytes and hold {cols} columns, "
                         f"got {qs[1]} and {ss[1]} bytes")
    return McAct8(q.data_ptr(), s.data_ptr(), rows, cols, qs[1], ss[1], code, 0)


def _act8_new(shape, rows, cols, fmt, dev):
    """An unset Act8 of checked arguments, and its structure."""
    q_ld = (cols + 15) & ~15
    s_ld = ((cols + ACT_BLOCK - 1) // ACT_BLOCK + 15) & ~15
    q = torch.empty(rows, q_ld, dtype=torch.uint8, device=dev)
    s = torch.empty(rows, s_ld, dtype=torch.uint8, device=dev)
    return Act8(q, s, shape, fmt), McAct8(q.data_ptr(), s.data_ptr(), rows, cols, q_ld, s_ld, _FMT[fmt], 0)


def act8_empty(shape, fmt: str = "int8", device=None) -> Act8:
    """An Act8 of this shape with unset contents."""
    _fmt_code(fmt)
    shape = tuple(int(n) for n in shape)
    if len(shape) < 1 or shape[-1] < 1 or min(shape) < 0:
        raise ValueError(f"shape must have at least one column, got {shape}")
    return _act8_new(shape, *_rows_cols(shape), fmt, device or "cuda")[0]


def act8_pack(x, fmt: str = "int8", *, out: Act8 = None, stream=None) -> Act8:
    """x (bf16 or fp32, any leading shape) in 8 bits (see mc_act8_pack).  ``out``:
    an Act8 of x's shape to write, whose own format then holds."""
    lib = load_library()
    _need_matrix(x, "x")
    code = _dtype_code(x)
    shape = tuple(x.shape)
    if out is None:
        _fmt_code(fmt)
        dev = x.device
    else:
        if tuple(out.shape) != shape:
            raise ValueError(f"out must have x's shape {shape}, got {tuple(out.shape)}")
        a = _act8_struct(out, "out")
        dev = _one_dev(x, out.q, out.scale)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        if out is None:
            out, a = _act8_new(shape, *_rows_cols(shape), fmt, dev)
        _check(lib.mc_act8_pack(x.data_ptr(), code, ctypes.byref(a), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return out


def act8_unpack(a: Act8, *, dtype=None, out=None, stream=None):
    """The values of an Act8 as bf16 (exact for whatever act8_pack or rms_norm wrote) or fp32."""
    lib = load_library()
    st = _act8_struct(a, "a")
    dev = _one_dev(a.q, a.scale, out)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        if out is None:
            out = torch.empty(*a.shape, dtype=dtype or torch.bfloat16, device=dev)
        else:
            _need_matrix(out, "out")
            if tuple(out.shape) != tuple(a.shape) or (dtype is not None and out.dtype != dtype):
                raise ValueError(f"out must have shape {tuple(a.shape)}" + (f" and type {dtype}" if dtype else ""))
        _check(lib.mc_act8_unpack(ctypes.byref(st), out.data_ptr(), _dtype_code(out), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return out


def rms_norm(x, weight, *, residual=None, eps: float = 1e-6, fmt: str = None, h_out=None, stream=None) -> RmsNorm:
    """Root-mean-square norm over the last dimension, with the residual's
    addition before it (see mc_rms_norm): h = x + residual (in x's type; x
    itself without), y = h * rstd * weight as bf16, or in 8 bits with ``fmt``.
    ``h_out`` may be x or residual itself."""
    lib = load_library()
    _need_matrix(x, "x")
    _need_cuda_contig(weight, "weight")
    shape = x.shape
    rows, cols = _rows_cols(shape)
    if weight.shape != (cols,):
        raise ValueError(f"weight must have shape ({cols},), got {tuple(weight.shape)}")
    if residual is not None:
        _need_like(residual, "residual", x, "x")
    if h_out is not None:
        _need_like(h_out, "h_out", x, "x")
    if h_out is not None and residual is None:
        raise ValueError("h_out goes with residual: without one, h is x")
    code, wcode = _dtype_code(x), _dtype_code(weight)
    if fmt is not None:
        _fmt_code(fmt)
    dev = _one_dev(x, weight, residual, h_out)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        if residual is not None and h_out is None:
            h_out = torch.empty_like(x)
        if fmt is None:
            y = torch.empty_like(x, dtype=torch.bfloat16)
            yp, y8 = y.data_ptr(), None
        else:
            y, st = _act8_new(tuple(shape), rows, cols, fmt, dev)
            yp, y8 = None, ctypes.byref(st)
        _check(lib.mc_rms_norm(x.data_ptr(), _ptr(residual), weight.data_ptr(), code, wcode, rows, cols, float(eps),
                               _ptr(h_out), yp, y8, rstd.data_ptr(), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return RmsNorm(x if residual is None else h_out, y, rstd)


def rms_norm_backward(dy, h, weight, rstd, *, dh=None, dx_out=None, workspace=None, stream=None):
    """(dx, dw) of ``rms_norm`` (see mc_rms_norm_backward): ``h`` is the tensor
    that rms_norm returned or its Act8, ``dh`` the gradient that reaches h past
    the norm.  dx is the gradient of x and of the residual; dw is fp32.
    ``dx_out`` may be dy or dh itself."""
    lib = load_library()
    _need_matrix(dy, "dy")
    _need_cuda_contig(weight, "weight")
    _need_cuda_contig(rstd, "rstd")
    rows, cols = _rows_cols(dy.shape)
    if weight.shape != (cols,):
        raise ValueError(f"weight must have shape ({cols},), got {tuple(weight.shape)}")
    if rstd.dtype != torch.float32 or rstd.numel() != rows:
        raise ValueError(f"rstd must be float32 with {rows} entries")
    if dh is not None:
        _need_like(dh, "dh", dy, "dy")
    if dx_out is not None:
        _need_like(dx_out, "dx_out", dy, "dy")
    if isinstance(h, Act8):
        if _rows_cols(h.shape) != (rows, cols):
            raise ValueError(f"h must have dy's shape {tuple(dy.shape)}, got {tuple(h.shape)}")
        st = _act8_struct(h, "h")
        hp, h8, held = None, ctypes.byref(st), (h.q, h.scale)
    else:
        _need_like(h, "h", dy, "dy")
        hp, h8, held = h.data_ptr(), None, (h,)
    code, wcode = _dtype_code(dy), _dtype_code(weight)
    dev = _one_dev(dy, weight, rstd, dh, dx_out, workspace, *held)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        dx = torch.empty_like(dy) if dx_out is None else dx_out
        dw = torch.empty(cols, dtype=torch.float32, device=dev)
        ws, nbytes = _scratch(workspace, lib.mc_rms_norm_backward_workspace_size(rows, cols), dev)
        _check(lib.mc_rms_norm_backward(dy.data_ptr(), _ptr(dh), hp, h8, weight.data_ptr(), rstd.data_ptr(), code, wcode,
                                        rows, cols, dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), nbytes, s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return dx, dw


def _scratch(workspace, need, dev):
    """The caller's workspace, or scratch from torch's allocator (ordered by the stream it is made on)."""
    if workspace is None:
        need = need or 16
        return torch.empty(need, dtype=torch.uint8, device=dev), need
    _need_cuda_contig(workspace, "workspace")
    return workspace, workspace.numel() * workspace.element_size()


def _grad_out(out, shape, dtype, accumulate, dev):
    if accumulate and out is None:
        raise ValueError("accumulate needs the sum to add to as out")
    if out is None:
        return torch.empty(*shape, dtype=dtype or torch.bfloat16, device=dev)
    _need_cuda_contig(out, "out")
    if tuple(out.shape) != tuple(shape) or (dtype is not None and out.dtype != dtype):
        raise ValueError(f"out must have shape {tuple(shape)}" + (f" and type {dtype}" if dtype else ""))
    return out


def _need_dy(dy):
    _need_matrix(dy, "dy")
    if dy.dtype != torch.bfloat16:
        raise TypeError("dy must be bfloat16")


def weight_grad(dy, x: Act8, *, dtype=None, out=None, accumulate: bool = False, workspace=None, stream=None):
    """The gradient [out-features, in-features] of an nn.Linear weight (see
    mc_weight_grad): dy^T x over all rows, dy bf16 [..., out-features], x the
    layer's input in 8 bits.  bf16 unless ``dtype`` or ``out`` say fp32; with
    ``accumulate`` it is added to ``out`` (fp32)."""
    lib = load_library()
    _need_dy(dy)
    st = _act8_struct(x, "x")
    rows, M = _rows_cols(dy.shape)
    if rows != st.rows:
        raise ValueError(f"dy and x must have the same rows, got {rows} and {st.rows}")
    dev = _one_dev(dy, x.q, x.scale, out, workspace)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        g = _grad_out(out, (M, st.cols), dtype, accumulate, dev)
        ws, nbytes = _scratch(workspace, lib.mc_weight_grad_workspace_size(rows, M, st.cols), dev)
        _check(lib.mc_weight_grad(dy.data_ptr(), ctypes.byref(st), M, g.data_ptr(), _dtype_code(g), int(bool(accumulate)),
                                  ws.data_ptr(), nbytes, s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return g


def _plan_part(t, name):
    if not (t.is_cuda and t.is_contiguous()):
        _need_cuda_contig(t, name)
    if t.dtype is not torch.int32:
        raise TypeError(f"{name} must be int32")


def _plan_pairs(plan):
    """(T, K) of the plan's ``position``, which is all that moving rows goes by."""
    pos = plan.position
    _plan_part(pos, "plan.position")
    shape = pos.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"plan.position must be 2D [T, K], got shape {tuple(shape)}")
    return shape


def expert_sort(idx, num_experts: int, *, workspace=None, stream=None) -> ExpertPlan:
    """The order of [T, K] (token, expert) pairs by expert (see mc_expert_sort):
    stable; an index outside [0, num_experts) drops its pair.  int32 or int64."""
    lib = load_library()
    _need_cuda_contig(idx, "idx")
    if idx.dtype not in (torch.int32, torch.int64):
        raise TypeError("idx must be int32 or int64")
    if idx.dim() != 2 or idx.shape[1] < 1:
        raise ValueError(f"idx must be 2D [T, K], got shape {tuple(idx.shape)}")
    T, K = int(idx.shape[0]), int(idx.shape[1])
    E = int(num_experts)
    dev = _one_dev(idx, workspace)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        # one allocation for the three results (each on a 16-byte boundary)
        n, o = -(-T * K // 4) * 4, -(-(max(E, 0) + 1) // 4) * 4
        buf = torch.empty(o + 2 * n, dtype=torch.int32, device=dev)
        plan = ExpertPlan(buf[:max(E, 0) + 1], buf[o:o + T * K], buf[o + n:o + n + T * K].view(T, K))
        ws, nbytes = _scratch(workspace, lib.mc_expert_sort_workspace_size(T, K, E), dev)
        _check(lib.mc_expert_sort(idx.data_ptr(), 64 if idx.dtype == torch.int64 else 32, T, K, E, plan.offsets.data_ptr(),
                                  plan.source.data_ptr(), plan.position.data_ptr(), ws.data_ptr(), nbytes, s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return plan


def _check_rows(t, name, rows, cols=None, dtype=None):
    _need_matrix(t, name)
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must have shape ({rows}, {'D' if cols is None else cols}), got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")


def _check_weights(w, T, K):
    _need_cuda_contig(w, "weights")
    if w.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if w.shape != (T, K):
        raise ValueError(f"weights must have shape {(T, K)}, got {tuple(w.shape)}")


def expert_gather(x, plan: ExpertPlan, *, out=None, stream=None):
    """Each token's row of x [T, D] (bf16 or fp32) at its pairs' sorted rows:
    [T * K, D].  Rows behind the last expert's are left as they are in ``out``,
    unset otherwise.  Its gradient is ``expert_combine`` without weights."""
    lib = load_library()
    T, K = _plan_pairs(plan)
    _check_rows(x, "x", T)
    code, D = _dtype_code(x), x.shape[1]
    dev = _one_dev(x, plan.position, out)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        if out is None:
            out = torch.empty(T * K, D, dtype=x.dtype, device=dev)
        else:
            _check_rows(out, "out", T * K, D, x.dtype)
        _check(lib.mc_expert_gather(x.data_ptr(), code, T, K, D, plan.position.data_ptr(), out.data_ptr(), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return out


def expert_combine(y, plan: ExpertPlan, weights=None, *, out=None, stream=None):
    """[T, D]: each token's sum of its pairs' rows of y [T * K, D], times
    weights [T, K] (fp32; none: ones), in fp32 and rounded once."""
    lib = load_library()
    T, K = _plan_pairs(plan)
    _check_rows(y, "y", T * K)
    if weights is not None:
        _check_weights(weights, T, K)
    code, D = _dtype_code(y), y.shape[1]
    dev = _one_dev(y, plan.position, weights, out)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        if out is None:
            out = torch.empty(T, D, dtype=y.dtype, device=dev)
        else:
            _check_rows(out, "out", T, D, y.dtype)
        _check(lib.mc_expert_combine(y.data_ptr(), code, T, K, D, plan.position.data_ptr(), _ptr(weights), out.data_ptr(), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return out


def expert_combine_backward(dout, y, plan: ExpertPlan, weights, *, out=None, stream=None):
    """(dy [T * K, D], dweights [T, K] fp32) of ``expert_combine`` with weights.
    Rows of dy behind the last expert's are left as they are in ``out``, unset
    otherwise; ``out`` may be y itself."""
    lib = load_library()
    T, K = _plan_pairs(plan)
    _check_rows(dout, "dout", T)
    code, D = _dtype_code(dout), dout.shape[1]
    _check_rows(y, "y", T * K, D, dout.dtype)
    _check_weights(weights, T, K)
    dev = _one_dev(dout, y, plan.position, weights, out)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        if out is None:
            out = torch.empty(T * K, D, dtype=y.dtype, device=dev)
        else:
            _check_rows(out, "out", T * K, D, y.dtype)
        dw = torch.empty(T, K, dtype=torch.float32, device=dev)
        _check(lib.mc_expert_combine_backward(dout.data_ptr(), y.data_ptr(), code, T, K, D, plan.position.data_ptr(),
                                              weights.data_ptr(), out.data_ptr(), dw.data_ptr(), s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return out, dw


def expert_weight_grad(dy, x: Act8, plan: ExpertPlan, *, gather: bool, dtype=None, out=None, accumulate: bool = False,
                       workspace=None, stream=None):
    """Gradients [E, out-features, in-features] of every expert's weight (see
    mc_expert_weight_grad) from dy bf16 [T * K, out-features] in sorted rows and
    x in 8 bits: in token order (``gather`` true: [T, in-features], e.g. the
    input of the experts' first products) or sorted like dy (``gather`` false).
    With ``gather``, pairs whose ``plan.position`` was set outside the rows after
    the sort add nothing, whatever their rows of dy hold; without, every row of
    an expert's range counts as it is."""
    lib = load_library()
    T, K = _plan_pairs(plan)
    _plan_part(plan.offsets, "plan.offsets")
    if plan.offsets.dim() != 1 or plan.offsets.shape[0] < 2:
        raise ValueError(f"plan.offsets must be 1D [E + 1], got shape {tuple(plan.offsets.shape)}")
    E = plan.offsets.shape[0] - 1
    _need_dy(dy)
    rows, M = _rows_cols(dy.shape)
    if rows != T * K:
        raise ValueError(f"dy must have T * K = {T * K} rows, got {rows}")
    st = _act8_struct(x, "x")
    if st.rows != (T if gather else rows):
        raise ValueError(f"x must have {T if gather else rows} rows, got {st.rows}")
    dev = _one_dev(dy, x.q, x.scale, plan.offsets, plan.position, out, workspace)
    on = _enter(dev, stream)
    try:
        s = _raw_stream(dev.index)
        g = _grad_out(out, (E, M, st.cols), dtype, accumulate, dev)
        ws, nbytes = _scratch(workspace, lib.mc_expert_weight_grad_workspace_size(rows, E, M, st.cols), dev)
        _check(lib.mc_expert_weight_grad(dy.data_ptr(), rows, ctypes.byref(st), plan.offsets.data_ptr(),
                                         plan.position.data_ptr() if gather else None, K, E, M, g.data_ptr(), _dtype_code(g),
                                         int(bool(accumulate)), ws.data_ptr(), nbytes, s))
    finally:
        if on is not None:
            on.__exit__(None, None, None)
    return g
