"""The routed experts beside the shared expert: routing, 8-bit block products, the experts' layer.

Thin bindings like the rest of the package (torch tensors in, the library's functions by name); formulas, layouts
and limits are in ``include/mse.h``.  8-bit tensors are ``torch.float8_e4m3fn`` (or ``uint8`` bit patterns) whose last
dimension is contiguous; their rows may have a pitch.  Rows whose pitch is a multiple of 16 bytes, as
``fp8_block_quantise`` makes them, take the tensor-core kernels.
"""
from __future__ import annotations


import moe_shared_expert_gb300 as _mse

_BLOCK = 128
_SCORING = {"softmax": 0, "sigmoid": 1}


def _torch():
    import torch
    return torch


def _blocks(n: int) -> int:
    return -(-n // _BLOCK)


def _pad16(n: int) -> int:
    return -(-n // 16) * 16


def _rows(t, name, dtypes, ndim):
    """A CUDA tensor whose last dimension is contiguous, and whose leading ones make rows of one pitch."""
    if t is None or not t.is_cuda or t.dtype not in dtypes or t.dim() != ndim:
        raise ValueError(f"{name}: need a {ndim}-d CUDA tensor of {dtypes}, got "
                         + ("None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"))
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension has to be contiguous, got strides {stride}")
    ld = stride[-2] if shape[-2] > 1 else max(shape[-1], stride[-2])
    if ld < shape[-1] or (ndim == 3 and shape[0] > 1 and stride[0] != shape[1] * ld):
        raise ValueError(f"{name}: rows of one pitch are needed, got shape {tuple(shape)}, strides {stride}")
    return ld


def _dense(t, name, dtype, shape):
    if t is None or not t.is_cuda or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous CUDA tensor of {dtype} {tuple(shape)}, got "
                         + ("None" if t is None else f"{t.dtype} {tuple(t.shape)} on {t.device}"))
    return t


def _e4m3():
    torch = _torch()
    return (torch.float8_e4m3fn, torch.uint8)


def _own_stream(t, stream):
    """Memory allocated here for a call on another stream than the current one stays taken until that call is done."""
    if stream is not None:
        torch = _torch()
        t.record_stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int) else stream)
    return t


def _empty(stream, shape, dtype, device):
    return _own_stream(_torch().empty(shape, dtype=dtype, device=device), stream)


# ---------------------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------------------

def moe_route(logits, top_k, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=2, renormalise=True,
              scale=1.0, ids=None, weights=None, stream=None):
    """(ids [T, top_k] int32, weights [T, top_k] fp32) of the router's logits [T, E] (bf16 or fp32).

    Experts are chosen by score + bias, best first, ties to the lower index; -inf, a type's lowest value and NaN
    close an expert.  Slots for which no expert is left hold id -1 and weight 0."""
    torch = _torch()
    ld = _rows(logits, "logits", (torch.bfloat16, torch.float32), 2)
    T, E = logits.shape
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}, got {scoring!r}")
    if bias is not None:
        _dense(bias, "bias", torch.float32, (E,))
    if ids is None:
        ids = _empty(stream, (T, max(top_k, 0)), torch.int32, logits.device)
    if weights is None:
        weights = _empty(stream, (T, max(top_k, 0)), torch.float32, logits.device)
    _dense(ids, "ids", torch.int32, (T, top_k))
    _dense(weights, "weights", torch.float32, (T, top_k))
    st = _mse.lib().moe_route(logits.data_ptr(), _mse._dtype_code(logits.dtype), T, E, ld, _mse._ptr(bias),
                              _SCORING[scoring], n_group, topk_group, group_top, top_k, int(bool(renormalise)),
                              scale, ids.data_ptr(), weights.data_ptr(), ids.numel(), _mse._stream(stream))
    _mse._check("moe_route", st)
    return ids, weights


# ---------------------------------------------------------------------------------------
# products in 8 bits
# ---------------------------------------------------------------------------------------

def fp8_block_quantise(x, block_rows=1, stream=None):
    """(q, scales): x [rows, K] or [n, rows, K] bf16 in e4m3 with a scale for each block of block_rows (1 or 128) x 128.

    q has x's shape and rows of a pitch of 16 bytes; scales is [.., ceil(rows / block_rows), ceil(K / 128)] fp32.
    A merged gate_up weight [E, 2I, H] is rounded as its halves, [2E, I, H], so that each half has its own blocks."""
    torch = _torch()
    if x is None or x.dim() not in (2, 3):
        raise ValueError("x: need a 2-d or 3-d tensor")
    _rows(x, "x", (torch.bfloat16,), x.dim())
    *lead, rows, K = x.shape
    q = _empty(stream, (*lead, rows, _pad16(K)), torch.uint8, x.device)
    scales = _empty(stream, (*lead, _blocks(rows) if block_rows != 1 else rows, _blocks(K)), torch.float32, x.device)
    for xm, qm, sm in [(x, q, scales)] if x.dim() == 2 else zip(x, q, scales):
        st = _mse.lib().fp8_block_quantise(xm.data_ptr(), rows, K, _rows(xm, "x", (torch.bfloat16,), 2), block_rows,
                                           qm.data_ptr(), qm.stride(0), qm.numel(), sm.data_ptr(), sm.numel(),
                                           _mse._stream(stream))
        _mse._check("fp8_block_quantise", st)
    return q.view(torch.float8_e4m3fn)[..., :K], scales


def fp8_block_matmul(xq, xs, wq, ws, out_dtype=None, out=None, stream=None):
    """out [T, N] = xq wq^T with block scales; xq [T, K], xs [T, K / 128], wq [N, K], ws [N / 128, K / 128]."""
    torch = _torch()
    ldx, ldw = _rows(xq, "xq", _e4m3(), 2), _rows(wq, "wq", _e4m3(), 2)
    (T, K), N = xq.shape, wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"xq and wq differ in K: {K} and {wq.shape[1]}")
    _dense(xs, "xs", torch.float32, (T, _blocks(K)))
    _dense(ws, "ws", torch.float32, (_blocks(N), _blocks(K)))
    code = _mse._dtype_code(out_dtype if out_dtype is not None else torch.bfloat16 if out is None else out.dtype)
    dtype = torch.float32 if code == _mse.F32 else torch.bfloat16
    if out is None:
        out = _empty(stream, (T, N), dtype, xq.device)
    _dense(out, "out", dtype, (T, N))
    st = _mse.lib().fp8_block_matmul(xq.data_ptr(), ldx, xs.data_ptr(), wq.data_ptr(), ldw, ws.data_ptr(), T, N, K,
                                     out.data_ptr(), code, out.numel(), _mse._stream(stream))
    _mse._check("fp8_block_matmul", st)
    return out


def fp8_linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(_mse.lib().fp8_block_linear_workspace_bytes(T, N, K))


def new_fp8_linear_workspace(T: int, N: int, K: int, device="cuda"):
    """A workspace for fp8_block_linear with up to T tokens."""
    return _torch().empty(max(fp8_linear_workspace_bytes(T, N, K), 256), dtype=_torch().uint8, device=device)


def fp8_block_linear(x, wq, ws, y_dtype=None, y=None, workspace=None, stream=None):
    """y [T, N] = x wq^T: x [T, K] bf16 is rounded to e4m3 in blocks of 1 x 128, wq and ws as in fp8_block_matmul."""
    torch = _torch()
    ldx, ldw = _rows(x, "x", (torch.bfloat16,), 2), _rows(wq, "wq", _e4m3(), 2)
    (T, K), N = x.shape, wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"x and wq differ in K: {K} and {wq.shape[1]}")
    _dense(ws, "ws", torch.float32, (_blocks(N), _blocks(K)))
    code = _mse._dtype_code(y_dtype if y_dtype is not None else torch.bfloat16 if y is None else y.dtype)
    dtype = torch.float32 if code == _mse.F32 else torch.bfloat16
    if y is None:
        y = _empty(stream, (T, N), dtype, x.device)
    _dense(y, "y", dtype, (T, N))
    if workspace is None:
        workspace = _own_stream(new_fp8_linear_workspace(T, N, K, x.device), stream)
    st = _mse.lib().fp8_block_linear(x.data_ptr(), ldx, wq.data_ptr(), ldw, ws.data_ptr(), T, N, K, y.data_ptr(),
                                     code, y.numel(), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), _mse._stream(stream))
    _mse._check("fp8_block_linear", st)
    return y


# ---------------------------------------------------------------------------------------
# the experts' layer
# ---------------------------------------------------------------------------------------

def moe_workspace_bytes(T: int, top_k: int, E: int, H: int, I: int) -> int:
    return int(_mse.lib().moe_experts_workspace_bytes(T, top_k, E, H, I))


def new_moe_workspace(T: int, top_k: int, E: int, H: int, I: int, device="cuda"):
    """A workspace for moe_experts_forward with up to T tokens."""
    return _torch().empty(max(moe_workspace_bytes(T, top_k, E, H, I), 256), dtype=_torch().uint8, device=device)


def moe_experts_forward(x, ids, weights, w_gate_up, s_gate_up, w_down, s_down, first_expert=0, shared=None, y=None,
                        workspace=None, stream=None):
    """y [T, H] = shared + the weighted sum of each token's routed experts that this rank holds.

    x [T, H] bf16; ids, weights [T, top_k] as moe_route gives them; w_gate_up [E, 2I, H] and w_down [E, H, I] in
    e4m3 with s_gate_up [E, 2 ceil(I / 128), ceil(H / 128)] (gate's blocks, then up's) and s_down
    [E, ceil(H / 128), ceil(I / 128)].  The rank holds experts first_expert .. first_expert + E - 1; pairs of other
    experts, and ids of -1, add nothing."""
    torch = _torch()
    _dense(x, "x", torch.bfloat16, x.shape if x is not None and x.dim() == 2 else (-1, -1))
    T, H = x.shape
    ld_gu, ld_dn = _rows(w_gate_up, "w_gate_up", _e4m3(), 3), _rows(w_down, "w_down", _e4m3(), 3)
    E, I = w_down.shape[0], w_down.shape[2]
    if tuple(w_gate_up.shape) != (E, 2 * I, H) or w_down.shape[1] != H:
        raise ValueError(f"w_gate_up {tuple(w_gate_up.shape)} and w_down {tuple(w_down.shape)} do not fit x "
                         f"{tuple(x.shape)}")
    _dense(s_gate_up, "s_gate_up", torch.float32, (E, 2 * _blocks(I), _blocks(H)))
    _dense(s_down, "s_down", torch.float32, (E, _blocks(H), _blocks(I)))
    k = ids.shape[1] if ids is not None and ids.dim() == 2 else -1
    _dense(ids, "ids", torch.int32, (T, k))
    _dense(weights, "weights", torch.float32, (T, k))
    if shared is not None:
        _dense(shared, "shared", torch.bfloat16, (T, H))
    if y is None:
        y = _empty(stream, (T, H), torch.bfloat16, x.device)
    _dense(y, "y", torch.bfloat16, (T, H))
    if workspace is None:
        workspace = _own_stream(new_moe_workspace(T, k, E, H, I, x.device), stream)
    st = _mse.lib().moe_experts_forward(x.data_ptr(), T, H, ids.data_ptr(), weights.data_ptr(), k,
                                        w_gate_up.data_ptr(), ld_gu, s_gate_up.data_ptr(), w_down.data_ptr(), ld_dn,
                                        s_down.data_ptr(), E, I, first_expert, _mse._ptr(shared), y.data_ptr(),
                                        y.numel(), workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(), _mse._stream(stream))
    _mse._check("moe_experts_forward", st)
    return y
