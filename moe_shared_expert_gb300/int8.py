"""Products in 8-bit integers: a scale for each token and each output channel, plain and by expert.

Thin bindings like the rest of the package; formulas, layouts and limits are in ``include/mse.h``.  All tensors of a call are on
the current device; outputs and workspaces lie apart from inputs and each other, but for y over x in ``int8_linear``.  8-bit
tensors are ``torch.int8`` whose last dimension is contiguous; rows of weights whose pitch is a
multiple of 16 bytes, as ``int8_quantise`` makes them, take the tensor-core kernels.

    wq, ws = int8_quantise(w)                      # once: a row of a weight is an output channel
    y = int8_linear(x, wq, ws)
    h, hs = int8_quantise(gate_up, swiglu=True)    # silu(gate) up
    y = int8_matmul(h, hs, wq_down, ws_down)

The sum over k is the integer itself, so results do not depend on which kernel ran.
"""
from __future__ import annotations

import ctypes

import moe_shared_expert_gb300 as _mse

from . import routed as _r
from . import rows as _s


def int8_workspace_bytes(T: int, N: int, K: int, groups: int = 1) -> int:
    return int(_mse.lib().int8_workspace_bytes(T, N, K, groups))


def new_int8_workspace(T: int, N: int, K: int, groups: int = 1, device="cuda"):
    """A workspace for int8_linear, int8_matmul and int8_grouped_matmul with up to T rows.

    Calls that run at the same time, captured graphs among them, need one each."""
    return _r._new_workspace(int8_workspace_bytes(T, N, K, groups), device)


def _space(workspace, stream, like, device, *sizes):
    if workspace is None:
        return _r._empty(stream, max(int8_workspace_bytes(*sizes), 256), _r.torch.uint8, like.device)
    _r._taken(workspace, device)
    return workspace


def int8_quantise(x, swiglu=False, offsets=None, q=None, scales=None, stream=None):
    """(q, scales): rows of x [rows, K] or [n, rows, K] (bf16 or fp32) in 8-bit integers with a scale each.

    With swiglu, x is [.., 2K] and silu(x[.., :K]) * x[.., K:] is rounded.  With offsets (as moe_sort gives them), rows from
    offsets[-1] on are left alone.  New q has rows of a pitch of 16 bytes."""
    torch = _s._ready() if _s._C is None else _r.torch
    if x is None or x.dim() not in (2, 3):
        raise ValueError(f"x: need a 2-d or 3-d tensor, got {_r._said(x)}")
    code, ld, (*lead, width), device = _s._floats(x, "x", x.dim())
    if swiglu and width % 2:
        raise ValueError(f"x: gate and up need an even number of columns, got {_r._said(x)}")
    K = width // 2 if swiglu else width
    rows = 1
    for n in lead:
        rows *= n
    last = None
    if offsets is not None:
        if offsets.dim() != 1 or offsets.shape[0] < 1 or len(lead) != 1:
            raise ValueError(f"offsets: need a 1-d tensor for a 2-d x, got {_r._said(offsets)}")
        _r._dense(offsets, "offsets", torch.int32, tuple(offsets.shape), device)
        last = offsets.data_ptr() + 4 * (offsets.shape[0] - 1)
    if q is None:
        q = _r._empty(stream, (*lead, _r._pad16(K)), torch.int8, x.device)[..., :K]
    ldq, shape, _ = _r._rows(q, "q", _s._I8, x.dim(), device)
    if tuple(shape) != (*lead, K):
        raise ValueError(f"q: need {(*lead, K)}, got {_r._said(q)}")
    if scales is None:
        scales = _r._empty(stream, tuple(lead), _s._F32, x.device)
    else:
        _r._dense(scales, "scales", _s._F32, tuple(lead), device)
    st = _s._C.int8_quantise(x.data_ptr(), code, rows, K, ld, 1 if swiglu else 0, last, q.data_ptr(), ldq, (rows - 1) * ldq + K,
                             scales.data_ptr(), _r._handle(stream, device))
    if st:
        _mse._check("int8_quantise", st)
    return q, scales


def int8_matmul(xq, xs, wq, ws, out_dtype=None, out=None, workspace=None, stream=None):
    """out [T, N] (bf16 unless out_dtype or out says fp32) = (xq wq^T) xs ws; xq [T, K], xs [T], wq [N, K], ws [N]."""
    if _s._C is None:
        _s._ready()
    ldx, (T, K), device = _r._rows(xq, "xq", _s._I8, 2)
    ldw, (N, Kw), _ = _r._rows(wq, "wq", _s._I8, 2, device)
    if K != Kw:
        raise ValueError(f"xq and wq differ in K: {K} and {Kw}")
    _r._dense(xs, "xs", _s._F32, (T,), device)
    _r._dense(ws, "ws", _s._F32, (N,), device)
    out, code = _s._out(out, out_dtype if out is not None or out_dtype is not None else _s._BF16, "out", (T, N), xq, stream, device)
    space = _space(workspace, stream, xq, device, T, N, K)
    st = _s._C.int8_matmul(xq.data_ptr(), ldx, xs.data_ptr(), wq.data_ptr(), ldw, ws.data_ptr(), T, N, K, out.data_ptr(), code,
                           T * N, space.data_ptr(), space.nbytes, _r._handle(stream, device))
    if st:
        _mse._check("int8_matmul", st)
    return out


def int8_grouped_matmul(xq, xs, offsets, wq, ws, out_dtype=None, out=None, workspace=None, stream=None):
    """out [T, N]: rows offsets[g] .. offsets[g + 1] of xq [T, K] times wq[g]^T; wq [G, N, K], ws [G, N], offsets [G + 1].

    Rows behind the last group's are left as they were."""
    torch = _s._ready() if _s._C is None else _r.torch
    ldx, (T, K), device = _r._rows(xq, "xq", _s._I8, 2)
    ldw, (G, N, Kw), _ = _r._rows(wq, "wq", _s._I8, 3, device)
    if K != Kw:
        raise ValueError(f"xq and wq differ in K: {K} and {Kw}")
    _r._dense(xs, "xs", _s._F32, (T,), device)
    _r._dense(ws, "ws", _s._F32, (G, N), device)
    _r._dense(offsets, "offsets", torch.int32, (G + 1,), device)
    out, code = _s._out(out, out_dtype if out is not None or out_dtype is not None else _s._BF16, "out", (T, N), xq, stream, device)
    space = _space(workspace, stream, xq, device, T, N, K, G)
    st = _s._C.int8_grouped_matmul(xq.data_ptr(), ldx, xs.data_ptr(), offsets.data_ptr(), G, wq.data_ptr(), ldw, ws.data_ptr(),
                                   T, N, K, out.data_ptr(), code, T * N, space.data_ptr(), space.nbytes,
                                   _r._handle(stream, device))
    if st:
        _mse._check("int8_grouped_matmul", st)
    return out


def int8_linear(x, wq, ws, y_dtype=None, y=None, workspace=None, stream=None):
    """y [T, N] = x wq^T: x [T, K] (bf16 or fp32) is rounded to 8-bit integers by rows, wq and ws as in int8_matmul."""
    if _s._C is None:
        _s._ready()
    x_code, ldx, (T, K), device = _s._floats(x, "x", 2)
    ldw, (N, Kw), _ = _r._rows(wq, "wq", _s._I8, 2, device)
    if K != Kw:
        raise ValueError(f"x and wq differ in K: {K} and {Kw}")
    _r._dense(ws, "ws", _s._F32, (N,), device)
    y, code = _s._out(y, y_dtype if y is not None or y_dtype is not None else _s._BF16, "y", (T, N), x, stream, device)
    space = _space(workspace, stream, x, device, T, N, K)
    st = _s._C.int8_linear(x.data_ptr(), x_code, ldx, wq.data_ptr(), ldw, ws.data_ptr(), T, N, K, y.data_ptr(), code, T * N,
                           space.data_ptr(), space.nbytes, _r._handle(stream, device))
    if st:
        _mse._check("int8_linear", st)
    return y


def int8_launch_plan(T: int, N: int, K: int, groups: int = 0) -> dict:
    """Kernel and split of a product (groups 0: plain) on the current device: see mse_int8_launch_plan in include/mse.h."""
    out = (ctypes.c_int32 * 4)()
    _mse._check("mse_int8_launch_plan", _mse.lib().mse_int8_launch_plan(T, N, K, groups, out))
    return dict(zip(("tile_rows", "parts", "one_launch"), map(int, out)))
