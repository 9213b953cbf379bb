"""Tokens sorted by expert and back with their weights, and the gradients of both ways.

For experts that a program runs itself: ``moe_route``'s ids sort the tokens' rows by expert, the experts take rows
``offsets[e] .. offsets[e + 1]`` each, and ``moe_unsort`` adds what they made of them for each token.  Thin bindings like the
rest of the package; formulas, layouts and limits are in ``include/mse.h``.  All tensors of a call are on the current device;
outputs and workspaces lie apart from inputs and each other, but for those that a call names.

Rows behind the last expert's (pairs of other ranks, or of padding, have none) are left as they were.  The gradients are calls
of their own, to be made from a program's backward pass:

    rows, place, offsets, _ = moe_sort(x, ids, E)
    y = moe_unsort(out, place, weights, base=shared)
    drows, dweights = moe_unsort_backward(dy, place, out, weights)     # base's gradient is dy
    dx = moe_sort_backward(dsorted, place)
"""
from __future__ import annotations

import ctypes
import os
import types

import moe_shared_expert_gb300 as _mse

from . import _build
from . import routed as _r

_NAMES = ("moe_sort", "moe_unsort", "moe_unsort_backward", "int8_quantise", "int8_matmul", "int8_grouped_matmul", "int8_linear")
_C = None   # the library's functions of these names, set with torch and the dtypes by _ready()


def _ready():
    """torch; what a call needs besides is looked up once, since a call's own Python is most of what a single token costs."""
    global _C, _BF16, _F32, _I8, _I32, _FLOATS
    if _r.torch is None:
        _r._load()
    if _C is None:
        _BF16, _F32, _I8, _I32 = _r.torch.bfloat16, _r.torch.float32, (_r.torch.int8,), _r.torch.int32
        _FLOATS = (_BF16, _F32)
        entries = {n: getattr(_mse.lib(), n) for n in _NAMES}
        if os.path.exists(_build.CALLS):   # the same functions without ctypes' conversions
            from . import _calls
            _calls.bind_rows(*(ctypes.cast(f, ctypes.c_void_p).value for f in entries.values()))
            entries = {n: getattr(_calls, n) for n in _NAMES}
        _C = types.SimpleNamespace(**entries)
    return _r.torch


def _floats(t, name, ndim, device=None):
    """(dtype code, row pitch, shape, device index) of rows in bf16 or fp32."""
    ld, shape, index = _r._rows(t, name, _FLOATS, ndim, device)
    return 1 if t.dtype is _F32 else 0, ld, shape, index


def _out(out, dtype, name, shape, like, stream, device):
    """The output tensor of a call, bf16 or fp32 (`dtype`, where there is no tensor yet), and its type's code."""
    if out is None:
        if dtype is not _BF16 and dtype is not _F32:
            raise ValueError(f"{name}: need bfloat16 or float32, got {dtype}")
        return _r._empty(stream, shape, dtype, like.device), 1 if dtype is _F32 else 0
    of = out.dtype
    if of is not _BF16 and of is not _F32 or dtype is not None and dtype is not of:
        raise ValueError(f"{name}: need a contiguous tensor of {dtype or _FLOATS} {tuple(shape)}, got {_r._said(out)}")
    _r._dense(out, name, of, shape, device)
    return out, 1 if of is _F32 else 0


def moe_sort_workspace_bytes(T: int, top_k: int, num_experts: int) -> int:
    return int(_mse.lib().moe_sort_workspace_bytes(T, top_k, num_experts))


def new_moe_sort_workspace(T: int, top_k: int, num_experts: int, device="cuda"):
    """A workspace for moe_sort with up to T tokens; calls that run at the same time, graphs among them, need one each."""
    return _r._new_workspace(moe_sort_workspace_bytes(T, top_k, num_experts), device)


def moe_sort(x, ids, num_experts, first_expert=0, scales=None, rows=None, row_scales=None, place=None, offsets=None,
             workspace=None, stream=None):
    """(rows [T * top_k, H], place [T, top_k], offsets [num_experts + 1], row_scales): x [T, H] sorted by expert.

    x holds values of 1, 2 or 4 bytes and is copied as it is; scales [T] fp32, where x has them, go along to row_scales
    [T * top_k] (else None).  ids [T, top_k] int32 as moe_route gives them; this rank's experts are first_expert ..
    first_expert + num_experts - 1, and place is -1 for pairs of others and for ids of -1.  New rows of 1-byte values have a
    pitch of 16 bytes."""
    torch = _ready() if _C is None else _r.torch
    if x is None or x.dtype.itemsize not in (1, 2, 4):
        raise ValueError(f"x: need values of 1, 2 or 4 bytes, got {_r._said(x)}")
    size = x.dtype.itemsize
    ldx, (T, H), device = _r._rows(x, "x", (x.dtype,), 2)
    if ids is None or ids.dim() != 2:
        raise ValueError(f"ids: need a 2-d tensor, got {_r._said(ids)}")
    k = ids.shape[1]
    _r._dense(ids, "ids", _I32, (T, k), device)
    if scales is not None:
        _r._dense(scales, "scales", _F32, (T,), device)
    elif row_scales is not None:
        raise ValueError("row_scales: there are no scales to sort")
    if rows is None:
        rows = _r._empty(stream, (T * k, _r._pad16(H) if size == 1 else H), x.dtype, x.device)[:, :H]
    ldr, shape, _ = _r._rows(rows, "rows", (x.dtype,), 2, device)
    if shape != (T * k, H):
        raise ValueError(f"rows: need {(T * k, H)}, got {_r._said(rows)}")
    if scales is not None:
        if row_scales is None:
            row_scales = _r._empty(stream, (T * k,), _F32, x.device)
        else:
            _r._dense(row_scales, "row_scales", _F32, (T * k,), device)
    if place is None:
        place = _r._empty(stream, (T, k), _I32, x.device)
    else:
        _r._dense(place, "place", _I32, (T, k), device)
    if offsets is None:
        offsets = _r._empty(stream, (max(num_experts, 0) + 1,), _I32, x.device)
    else:
        _r._dense(offsets, "offsets", _I32, (num_experts + 1,), device)
    if workspace is None:
        workspace = _r._empty(stream, max(moe_sort_workspace_bytes(T, k, num_experts), 256), torch.uint8, x.device)
    else:
        _r._taken(workspace, device)
    st = _C.moe_sort(x.data_ptr(), size, T, H, ldx, ids.data_ptr(), k, num_experts, first_expert,
                     None if scales is None else scales.data_ptr(), rows.data_ptr(), ldr, (T * k - 1) * ldr + H,
                     None if row_scales is None else row_scales.data_ptr(), place.data_ptr(), offsets.data_ptr(),
                     workspace.data_ptr(), workspace.nbytes, _r._handle(stream, device))
    if st:
        _mse._check("moe_sort", st)
    return rows, place, offsets, row_scales


def moe_unsort(rows, place, weights=None, base=None, y_dtype=None, y=None, stream=None):
    """y [T, H] = base + sum over j of weights[t, j] rows[place[t, j]], in fp32, rounded once.

    rows [n, H] and y are bf16 or fp32 (y: rows' type unless y_dtype or y says otherwise), place [T, top_k] as moe_sort gives
    it, weights [T, top_k] fp32 (None: 1), base [T, H] of y's type (None: 0; y itself is allowed)."""
    if _C is None:
        _ready()
    code, ldr, (n, H), device = _floats(rows, "rows", 2)
    if place is None or place.dim() != 2:
        raise ValueError(f"place: need a 2-d tensor, got {_r._said(place)}")
    T, k = place.shape
    _r._dense(place, "place", _I32, (T, k), device)
    if weights is not None:
        _r._dense(weights, "weights", _F32, (T, k), device)
    y, y_code = _out(y, y_dtype if y_dtype is not None or y is not None else rows.dtype, "y", (T, H), rows, stream, device)
    if base is not None:
        _r._dense(base, "base", y.dtype, (T, H), device)
    st = _C.moe_unsort(rows.data_ptr(), code, n, ldr, place.data_ptr(), None if weights is None else weights.data_ptr(), T, H, k,
                       None if base is None else base.data_ptr(), y.data_ptr(), y_code, T * H, _r._handle(stream, device))
    if st:
        _mse._check("moe_unsort", st)
    return y


def moe_unsort_backward(dy, place, rows=None, weights=None, drows=None, dweights=None, rows_count=None, stream=None):
    """(drows [n, H], dweights [T, top_k]): moe_unsort's gradients from dy [T, H]; base's is dy itself.

    rows and weights as moe_unsort had them.  Without weights, drows alone (dweights None): rows is not needed, and drows has
    the shape of `drows`, or rows_count (default T * top_k) rows of dy's type.  Rows that are no pair's place are left as they
    were.  drows may be rows, and dweights weights."""
    if _C is None:
        _ready()
    dy_code, ld, (T, H), device = _floats(dy, "dy", 2)
    if ld != H and T > 1:
        raise ValueError(f"dy: need a contiguous tensor, got {_r._said(dy)}")
    if place is None or place.dim() != 2:
        raise ValueError(f"place: need a 2-d tensor, got {_r._said(place)}")
    k = place.shape[1]
    _r._dense(place, "place", _I32, (T, k), device)
    if weights is not None:
        _r._dense(weights, "weights", _F32, (T, k), device)
        if rows is None:
            raise ValueError("rows: needed for the weights' gradient")
        if dweights is None:
            dweights = _r._empty(stream, (T, k), _F32, dy.device)
        else:
            _r._dense(dweights, "dweights", _F32, (T, k), device)
    elif dweights is not None:
        raise ValueError("dweights: there are no weights")
    code, ldr, n = None, 0, rows_count if rows_count is not None else T * k
    if rows is not None:
        code, ldr, (n, Hr), _ = _floats(rows, "rows", 2, device)
        if Hr != H:
            raise ValueError(f"rows and dy differ in H: {Hr} and {H}")
    if drows is None:
        drows = _r._empty(stream, (n, H), dy.dtype if rows is None else rows.dtype, dy.device)
    d_code, ldd, (nd, Hd), _ = _floats(drows, "drows", 2, device)
    if Hd != H or (code is not None and (d_code != code or nd != n)) or (rows_count is not None and nd != n):
        raise ValueError(f"drows: need {(n, H)} like rows, got {_r._said(drows)}")
    st = _C.moe_unsort_backward(dy.data_ptr(), dy_code, place.data_ptr(), None if weights is None else weights.data_ptr(),
                                None if rows is None else rows.data_ptr(), d_code, ldr, nd, T, H, k, drows.data_ptr(), ldd,
                                (nd - 1) * ldd + H, None if dweights is None else dweights.data_ptr(), _r._handle(stream, device))
    if st:
        _mse._check("moe_unsort_backward", st)
    return drows, dweights


def moe_sort_backward(drows, place, dx_dtype=None, dx=None, stream=None):
    """dx [T, H] = sum over j of drows[place[t, j]]: moe_sort's gradient, in fp32, rounded once."""
    return moe_unsort(drows, place, y_dtype=dx_dtype, y=dx, stream=stream)
