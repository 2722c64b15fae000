"""Tokens sorted by expert and back, for device tensors, and a layer of int8
experts built from them.  Argument marshalling only, as ``binding``; the
definitions are those of ``include/dgemm.h``.

A pair is one choice of one token: T tokens with k choices each make T*k
pairs, in token order.  ``slot`` [T, k] holds each pair's row in the order
sorted by expert (-1: dropped).
"""

from __future__ import annotations

from .quantized import call, matmul_grouped, one_device, pitch, quantize_i8, takes_stream, type_code
from .binding import load_library


@takes_stream
def expert_sort(ids, experts, with_token=False):
    """Stable sort of the pairs by expert.

    ids: int64 or int32, [T, k], contiguous (a router's topk indices); an id
    outside 0 .. experts - 1 drops its pair.  Returns (offsets [experts + 1],
    slot [T, k], pair [T*k]), all int32: where each expert's rows begin, each
    pair's row, and each row's pair (-1 behind the last); ``with_token`` adds
    each row's token [T*k], the ``row_index`` of ``matmul_grouped``.
    """
    import torch
    device = one_device("ids", ids)
    if ids.dtype not in (torch.int64, torch.int32):
        raise TypeError("ids must be int64 or int32")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be contiguous, one row of choices for each token")
    T, k = ids.shape
    n = T * k
    if not 0 <= experts < 2 ** 31:
        raise ValueError("experts must be a count")
    # One allocation for all results.
    buf = torch.empty((experts + 1 + (3 if with_token else 2) * n,), dtype=torch.int32, device=device)
    at = experts + 1
    offsets, slot = buf.as_strided((at,), (1,)), buf.as_strided((T, k), (k, 1), at)
    pair = buf.as_strided((n,), (1,), at + n)
    token = buf.as_strided((n,), (1,), at + 2 * n) if with_token else None
    need = load_library().expert_sort_workspace(T, k, experts)
    ws = torch.empty((need,), dtype=torch.uint8, device=device) if need > 0 else None
    call("expert_sort", device, T, k, experts, ids.data_ptr(), ids.element_size(), offsets.data_ptr(),
         slot.data_ptr(), pair.data_ptr(), token.data_ptr() if with_token else None,
         ws.data_ptr() if ws is not None else None, max(need, 0))
    return (offsets, slot, pair, token) if with_token else (offsets, slot, pair)


def _slots(slot):
    import torch
    if slot.dtype != torch.int32 or slot.dim() != 2 or not slot.is_contiguous():
        raise TypeError("slot must be a contiguous int32 tensor, one row for each token")
    return slot.shape


def _weights(weights, slot):
    import torch
    if weights is None:
        return None
    if weights.dtype != torch.float32 or weights.shape != slot.shape or not weights.is_contiguous():
        raise TypeError("weights must be a contiguous float32 tensor of slot's shape")
    return weights.data_ptr()


def _rows(t, what, rows, H, dtype):
    if t.dim() != 2 or t.shape[1] != H or (rows is not None and t.shape[0] != rows) or t.dtype != dtype:
        raise ValueError(f"{what} must be a {dtype} tensor of shape ({'rows' if rows is None else rows}, {H})")
    return pitch(t, what)


@takes_stream
def expert_dispatch(x, slot, out=None, rows=None):
    """Rows to their sorted places: ``out[slot[t, j]] = x[t]``.  x: [T, H],
    float32, float16 or bfloat16.  A new out has ``rows`` (default T*k) rows;
    rows that no slot names are not written.  No slot may occur twice."""
    import torch
    device = one_device("x, slot and out", x, slot, out)
    T, k = _slots(slot)
    code = type_code(x.dtype)
    H = x.shape[-1]
    ldx = _rows(x, "x", T, H, x.dtype)
    if out is None:
        out, ldy = torch.empty((T * k if rows is None else rows, H), dtype=x.dtype, device=device), H
    else:
        ldy = _rows(out, "out", rows, H, x.dtype)
    call("expert_dispatch", device, T, k, H, code, x.data_ptr(), ldx, slot.data_ptr(), out.data_ptr(),
         out.shape[0], ldy)
    return out


@takes_stream
def expert_combine(y, slot, weights=None, out=None):
    """Sorted rows back to their tokens: ``out[t] = sum_j weights[t, j] *
    y[slot[t, j]]`` in float32, rounded once to y's dtype (weights None: all
    1).  A token with no pair left gets zeros."""
    import torch
    device = one_device("y, slot, weights and out", y, slot, weights, out)
    T, k = _slots(slot)
    code = type_code(y.dtype)
    H = y.shape[-1]
    ldy = _rows(y, "y", None, H, y.dtype)
    w = _weights(weights, slot)
    if out is None:
        out, ldo = torch.empty((T, H), dtype=y.dtype, device=device), H
    else:
        ldo = _rows(out, "out", T, H, y.dtype)
    call("expert_combine", device, T, k, H, code, y.data_ptr(), y.shape[0], ldy, slot.data_ptr(), w,
         out.data_ptr(), ldo)
    return out


@takes_stream
def expert_dispatch_grad(dy, slot, out=None):
    """The gradient of ``expert_dispatch``: ``dx[t] = sum_j dy[slot[t, j]]``."""
    return expert_combine(dy, slot, None, out=out)


@takes_stream
def expert_combine_grad(dout, y, slot, weights=None, dy=None, dweights=None):
    """The gradients of ``expert_combine``: (dy, dweights) with
    ``dy[slot[t, j]] = weights[t, j] * dout[t]`` (rows that no slot names are
    not written) and ``dweights[t, j] = dout[t] . y[slot[t, j]]`` (float32, 0
    for a dropped pair).  dy must not overlap y or dout; no slot may occur
    twice."""
    import torch
    device = one_device("dout, y, slot, weights, dy and dweights", dout, y, slot, weights, dy, dweights)
    T, k = _slots(slot)
    code = type_code(y.dtype)
    H = y.shape[-1]
    ldy = _rows(y, "y", None, H, y.dtype)
    ldo = _rows(dout, "dout", T, H, y.dtype)
    w = _weights(weights, slot)
    if dy is None:
        dy, lddy = torch.empty((y.shape[0], H), dtype=y.dtype, device=device), H
    else:
        lddy = _rows(dy, "dy", y.shape[0], H, y.dtype)
    if dweights is None:
        dweights = torch.empty((T, k), dtype=torch.float32, device=device)
    elif dweights.dtype != torch.float32 or dweights.shape != slot.shape or not dweights.is_contiguous():
        raise TypeError("dweights must be a contiguous float32 tensor of slot's shape")
    call("expert_combine_grad", device, T, k, H, code, dout.data_ptr(), ldo, y.data_ptr(), y.shape[0], ldy,
         slot.data_ptr(), w, dy.data_ptr(), lddy, dweights.data_ptr())
    return dy, dweights


@takes_stream
def matmul_experts(x, ids, weights, b, scale_b, out=None):
    """One linear layer of int8 experts: ``out[t] = sum_j weights[t, j] *
    (b[e] @ x[t])``, e = ids[t, j], with x quantised to int8 row by row.
    Each product is rounded to x's type before its weight is applied (as a
    sequence of layers would; one past float16's range is an infinity), the
    weighted sum once more.

    x: [T, K], float32, float16 or bfloat16 (and so the result, [T, N]); ids,
    weights: [T, k]; b: int8, experts x N x K with scale_b experts x N, as
    ``matmul_grouped`` takes them.  Each token is quantised once; the products
    read its row through the sort, so no sorted copy of x is made.  T times K
    (rounded up to 16) has to stay below 2^31.
    """
    one_device("x, ids, weights, b, scale_b and out", x, ids, weights, b, scale_b, out)
    if x.dim() != 2 or ids.dim() != 2 or x.shape[0] != ids.shape[0]:
        raise ValueError(f"x {tuple(x.shape)} and ids {tuple(ids.shape)} must have one row for each token")
    if b.dim() != 3 or x.shape[1] != b.shape[2]:
        raise ValueError(f"x {tuple(x.shape)} and b {tuple(b.shape)} do not chain")
    q, scale = quantize_i8(x)
    offsets, slot, _, token = expert_sort(ids, b.shape[0], with_token=True)
    y = matmul_grouped(q, b, offsets, scale, scale_b, out_dtype=x.dtype, row_index=token)
    return expert_combine(y, slot, weights, out=out)
