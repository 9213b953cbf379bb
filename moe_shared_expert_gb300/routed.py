"""The routed experts beside the shared expert: routing, 8-bit block products, the experts' layer.

Thin bindings like the rest of the package (torch tensors in, the library's functions by name); formulas, layouts
and limits are in ``include/mse.h``.  All tensors of a call are on the current device.  8-bit tensors are
``torch.float8_e4m3fn`` (or ``uint8`` bit patterns) whose last dimension is contiguous; their rows may have a pitch.
Rows whose pitch is a multiple of 16 bytes, as ``fp8_block_quantise`` makes them, take the tensor-core kernels.
"""
from __future__ import annotations

import ctypes
import os

import moe_shared_expert_gb300 as _mse

from . import _build

_BLOCK = 128
_SCORING = {"softmax": 0, "sigmoid": 1}
torch = None   # set by _load(); the package itself imports without it


def _load():
    """torch, the library's functions and the dtypes, looked up once: a call's own Python is most of what a
    single token's operators cost."""
    global torch, _C, _BF16, _F32, _E4M3, _raw_stream, _current, _call_route, _call_linear, _call_matmul, _call_experts
    import torch as _torch
    _C = C = _mse.lib()
    entries = C.moe_route, C.fp8_block_linear, C.fp8_block_matmul, C.moe_experts_forward
    _call_route, _call_linear, _call_matmul, _call_experts = entries
    if os.path.exists(_build.CALLS):   # the same functions without ctypes' conversions
        from . import _calls
        _calls.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in entries))
        _call_route, _call_linear = _calls.moe_route, _calls.fp8_block_linear
        _call_matmul, _call_experts = _calls.fp8_block_matmul, _calls.moe_experts_forward
    _BF16, _F32, _E4M3 = _torch.bfloat16, _torch.float32, (_torch.float8_e4m3fn, _torch.uint8)
    # the current stream's handle without making a Stream object, where this torch has it
    _raw_stream = getattr(_torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: _torch.cuda.current_stream(index).cuda_stream)
    _current = getattr(_torch._C, "_cuda_getDevice", None) or _torch.cuda.current_device
    torch = _torch


def _blocks(n: int) -> int:
    return -(-n // _BLOCK)


def _pad16(n: int) -> int:
    return -(-n // 16) * 16


def _said(t):
    return "None" if t is None else f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}"


def _rows(t, name, dtypes, ndim, device=None):
    """(pitch of the rows, shape, index of the GPU) of a tensor whose last dimension is contiguous and whose matrices follow
    one another.  It is on `device`; a call's first operand, without one, on the current device: the library launches there."""
    index = -1 if t is None else t.get_device()
    if index < 0 or t.dtype not in dtypes or t.dim() != ndim:
        raise ValueError(f"{name}: need a {ndim}-d CUDA tensor of {dtypes}, got {_said(t)}")
    if index != (_current() if device is None else device):
        raise ValueError(f"{name}: on cuda:{index}, and not on the call's device, cuda:{_current() if device is None else device}")
    shape, stride = t.shape, t.stride()
    cols = shape[-1]
    ld = stride[-2] if shape[-2] > 1 else max(cols, stride[-2])
    if (cols > 1 and stride[-1] != 1) or ld < cols or (ndim == 3 and shape[0] > 1 and stride[0] != shape[1] * ld):
        raise ValueError(f"{name}: contiguous rows of one pitch are needed, got {_said(t)}")
    return ld, shape, index


def _dense(t, name, dtype, shape, device):
    if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous tensor of {dtype} {tuple(shape)} on cuda:{device}, got {_said(t)}")


def _taken(workspace, device):
    """A caller's workspace: its bytes are what the call may write."""
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: need a contiguous tensor on cuda:{device}, got {_said(workspace)}")


def _handle(stream, device):
    """cudaStream_t of `stream`, or of the device's current stream."""
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(stream, shape, dtype, device):
    """New memory for a call on `stream`.

    Another stream than the current one fills its own blocks: one that the current stream has let go may still be in
    use by its kernels.  And what the caller drops is not taken again before the current stream, too, is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):   # (0 is the default stream's handle, and would make a new stream)
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


# ---------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------

def moe_route(logits, top_k, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2, renormalise=True,
              scale=1.0, ids=None, weights=None, stream=None):
    """(ids [T, top_k] int32, weights [T, top_k] fp32) of the router's logits [T, E] (bf16 or fp32).

    Experts are chosen by score + bias, best first, ties to the lower index; -inf, a type's lowest value and NaN
    close an expert.  Slots for which no expert is left hold id -1 and weight 0."""
    if torch is None:
        _load()
    ld, (T, E), device = _rows(logits, "logits", (_BF16, _F32), 2)
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    if bias is not None:
        _dense(bias, "bias", _F32, (E,), device)
    if ids is None:
        ids = _empty(stream, (T, max(top_k, 0)), torch.int32, logits.device)
    else:
        _dense(ids, "ids", torch.int32, (T, top_k), device)
    if weights is None:
        weights = _empty(stream, (T, max(top_k, 0)), _F32, logits.device)
    else:
        _dense(weights, "weights", _F32, (T, top_k), device)
    st = _call_route(logits.data_ptr(), int(logits.dtype is _F32), T, E, ld, None if bias is None else bias.data_ptr(),
                      _SCORING[scoring], n_group, topk_group, group_top, top_k, 1 if renormalise else 0, scale,
                      ids.data_ptr(), weights.data_ptr(), T * top_k, _handle(stream, device))
    if st:
        _mse._check("moe_route", st)
    return ids, weights


# ---------------------------------------------------------------------------------------
# products in 8 bits
# ---------------------------------------------------------------------------------------

def fp8_block_quantise(x, block_rows=1, stream=None):
    """(q, scales): x [rows, K] or [n, rows, K] bf16 in e4m3 with a scale for each block of block_rows (1 or 128) x 128.

    q has x's shape and rows of a pitch of 16 bytes; scales is [.., ceil(rows / block_rows), ceil(K / 128)] fp32.
    A merged gate_up weight [E, 2I, H] is rounded as its halves, [2E, I, H], so that each half has its own blocks."""
    if torch is None:
        _load()
    if x is None or x.dim() not in (2, 3):
        raise ValueError(f"x: need a 2-d or 3-d tensor, got {_said(x)}")
    ld, (*lead, rows, K), device = _rows(x, "x", (_BF16,), x.dim())
    pitch, srows, kb = _pad16(K), rows if block_rows == 1 else _blocks(rows), _blocks(K)
    q = _empty(stream, (*lead, rows, pitch), torch.uint8, x.device)
    scales = _empty(stream, (*lead, srows, kb), _F32, x.device)
    for i in range(lead[0] if lead else 1):
        st = _C.fp8_block_quantise(x.data_ptr() + 2 * i * rows * ld, rows, K, ld, block_rows,
                                   q.data_ptr() + i * rows * pitch, pitch, rows * pitch,
                                   scales.data_ptr() + 4 * i * srows * kb, srows * kb, _handle(stream, device))
        if st:
            _mse._check("fp8_block_quantise", st)
    return q.view(torch.float8_e4m3fn)[..., :K], scales


def _out(out, dtype, name, shape, like, stream):
    """The output tensor of a product and its type's code."""
    code = _mse._dtype_code(dtype if dtype is not None else _BF16 if out is None else out.dtype)
    dtype = _F32 if code else _BF16
    if out is None:
        return _empty(stream, shape, dtype, like.device), code
    _dense(out, name, dtype, shape, like.get_device())
    return out, code


def fp8_block_matmul(xq, xs, wq, ws, out_dtype=None, out=None, stream=None):
    """out [T, N] = xq wq^T with block scales; xq [T, K], xs [T, K / 128], wq [N, K], ws [N / 128, K / 128]."""
    if torch is None:
        _load()
    ldx, (T, K), device = _rows(xq, "xq", _E4M3, 2)
    ldw, (N, Kw), _ = _rows(wq, "wq", _E4M3, 2, device)
    if K != Kw:
        raise ValueError(f"xq and wq differ in K: {K} and {Kw}")
    _dense(xs, "xs", _F32, (T, _blocks(K)), device)
    _dense(ws, "ws", _F32, (_blocks(N), _blocks(K)), device)
    out, code = _out(out, out_dtype, "out", (T, N), xq, stream)
    st = _call_matmul(xq.data_ptr(), ldx, xs.data_ptr(), wq.data_ptr(), ldw, ws.data_ptr(), T, N, K,
                             out.data_ptr(), code, T * N, _handle(stream, device))
    if st:
        _mse._check("fp8_block_matmul", st)
    return out


def fp8_linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(_mse.lib().fp8_block_linear_workspace_bytes(T, N, K))


def _new_workspace(nbytes, device):
    if torch is None:
        _load()
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def new_fp8_linear_workspace(T: int, N: int, K: int, device="cuda"):
    """A workspace for fp8_block_linear with up to T tokens."""
    return _new_workspace(fp8_linear_workspace_bytes(T, N, K), device)


def fp8_block_linear(x, wq, ws, y_dtype=None, y=None, workspace=None, stream=None):
    """y [T, N] = x wq^T: x [T, K] bf16 is rounded to e4m3 in blocks of 1 x 128, wq and ws as in fp8_block_matmul."""
    if torch is None:
        _load()
    ldx, (T, K), device = _rows(x, "x", (_BF16,), 2)
    ldw, (N, Kw), _ = _rows(wq, "wq", _E4M3, 2, device)
    if K != Kw:
        raise ValueError(f"x and wq differ in K: {K} and {Kw}")
    _dense(ws, "ws", _F32, (_blocks(N), _blocks(K)), device)
    y, code = _out(y, y_dtype, "y", (T, N), x, stream)
    if workspace is None:
        workspace = _empty(stream, max(fp8_linear_workspace_bytes(T, N, K), 256), torch.uint8, x.device)
    else:
        _taken(workspace, device)
    st = _call_linear(x.data_ptr(), ldx, wq.data_ptr(), ldw, ws.data_ptr(), T, N, K, y.data_ptr(), code, T * N,
                             workspace.data_ptr(), workspace.nbytes, _handle(stream, device))
    if st:
        _mse._check("fp8_block_linear", st)
    return y


# ---------------------------------------------------------------------------------------
# the experts' layer
# ---------------------------------------------------------------------------------------

def moe_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(_mse.lib().moe_experts_workspace_bytes(T, top_k, E, H, I))


def new_moe_workspace(T: int, top_k: int, E: int, H: int, I: int, device="cuda"):
    """A workspace for moe_experts_forward with up to T tokens."""
    return _new_workspace(moe_workspace_bytes(T, top_k, E, H, I), device)


def moe_experts_forward(x, ids, weights, w_gate_up, s_gate_up, w_down, s_down, first_expert=0, shared=None, y=None,
                        workspace=None, stream=None):
    """y [T, H] = shared + the weighted sum of each token's routed experts that this rank holds.

    x [T, H] bf16; ids, weights [T, top_k] as moe_route gives them; w_gate_up [E, 2I, H] and w_down [E, H, I] in
    e4m3 with s_gate_up [E, 2 ceil(I / 128), ceil(H / 128)] (gate's blocks, then up's) and s_down
    [E, ceil(H / 128), ceil(I / 128)].  The rank holds experts first_expert .. first_expert + E - 1; pairs of other
    experts, and ids of -1, add nothing."""
    if torch is None:
        _load()
    ld_gu, of_gate_up, device = _rows(w_gate_up, "w_gate_up", _E4M3, 3)
    ld_dn, (E, H, I), _ = _rows(w_down, "w_down", _E4M3, 3, device)
    if of_gate_up != (E, 2 * I, H):
        raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} does not fit w_down {tuple(w_down.shape)}")
    if x is None or ids is None or x.dim() != 2 or ids.dim() != 2:
        raise ValueError(f"x and ids: need 2-d tensors, got {_said(x)} and {_said(ids)}")
    T, k = ids.shape
    hb, ib = _blocks(H), _blocks(I)
    _dense(x, "x", _BF16, (T, H), device)
    _dense(ids, "ids", torch.int32, (T, k), device)
    _dense(weights, "weights", _F32, (T, k), device)
    _dense(s_gate_up, "s_gate_up", _F32, (E, 2 * ib, hb), device)
    _dense(s_down, "s_down", _F32, (E, hb, ib), device)
    if shared is not None:
        _dense(shared, "shared", _BF16, (T, H), device)
    if y is None:
        y = _empty(stream, (T, H), _BF16, x.device)
    else:
        _dense(y, "y", _BF16, (T, H), device)
    if workspace is None:
        workspace = _empty(stream, max(moe_workspace_bytes(T, k, E, H, I), 256), torch.uint8, x.device)
    else:
        _taken(workspace, device)
    st = _call_experts(x.data_ptr(), T, H, ids.data_ptr(), weights.data_ptr(), k, w_gate_up.data_ptr(), ld_gu,
                                s_gate_up.data_ptr(), w_down.data_ptr(), ld_dn, s_down.data_ptr(), E, I, first_expert,
                                None if shared is None else shared.data_ptr(), y.data_ptr(), T * H,
                                workspace.data_ptr(), workspace.nbytes, _handle(stream, device))
    if st:
        _mse._check("moe_experts_forward", st)
    return y


# ---------------------------------------------------------------------------------------
# what a call would launch
# ---------------------------------------------------------------------------------------

def _plan(func, keys, *sizes):
    out = (ctypes.c_int32 * 8)()
    _mse._check(func, getattr(_mse.lib(), func)(*sizes, out))
    return dict(zip(keys, map(int, out)))


def fp8_launch_plan(T: int, N: int, K: int) -> dict:
    """Kernel and split of a product on the current device: see mse_fp8_launch_plan in include/mse.h."""
    return _plan("mse_fp8_launch_plan", ("tile_rows", "parts", "ctas", "one_launch"), T, N, K)


def moe_launch_plan(T: int, top_k: int, E: int, H: int, I: int) -> dict:
    """Kernels and splits of the experts' layer on the current device: see mse_moe_launch_plan in include/mse.h."""
    return _plan("mse_moe_launch_plan", ("tile_rows", "gate_up_parts", "gate_up_ctas", "down_parts", "down_ctas",
                                         "tiles_from_ids", "counted_apart"), T, top_k, E, H, I)
