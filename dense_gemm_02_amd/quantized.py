"""8-bit integer linear layers for device tensors: rows to int8, the int8
product with scales for each token and channel, and the products of a mixture
of experts over sorted tokens.  Argument marshalling only, as ``binding``; the
definitions are those of ``include/dgemm.h``.

Every function takes the keyword ``stream`` (a torch stream or a raw handle;
default: the current stream of the tensors' device) and runs on the tensors'
device, whichever is current.
"""

from __future__ import annotations

import functools

from .binding import DgemmError, _factor_vector, _need, load_library

# What a call needs of torch and the library, looked up once: on a small call
# the lookups would cost as much as its launch.
_TYPES = {}
_calls = {}
_raw_stream = _current_device = None


def type_code(dtype):
    """The dgemm_type of a torch dtype."""
    if not _TYPES:
        import torch
        _TYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    code = _TYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}: float32, float16 or bfloat16")
    return code


def _entry(name):
    global _raw_stream, _current_device
    import torch
    # (The raw handle: building a Stream object alone takes 1.7 us.)
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _calls[name] = getattr(load_library(), name)
    return _calls[name]


def call(name, device, *args):
    """One library call on the current stream of `device`, with it current."""
    fn = _calls.get(name) or _entry(name)
    index = device.index
    if index == _current_device():
        st = fn(*args, _raw_stream(index))
    else:
        import torch
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        raise DgemmError(st, name)


def takes_stream(fn):
    """Gives fn a keyword ``stream`` (a torch stream or a raw handle): the
    call, and what it allocates, then belong to that stream, as under ``with
    torch.cuda.stream(stream)``; inputs have to be ready on it."""
    @functools.wraps(fn)
    def with_stream(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        # (Any tensor tells: keywords come in any order, None and numbers among them.)
        device = one_device("the arguments", next((t for t in (*args, *kw.values()) if hasattr(t, "is_cuda")), None))
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return with_stream


def one_device(names, first, *rest):
    """All of them device tensors of one device (None: not given)."""
    if not getattr(first, "is_cuda", False):
        raise TypeError(f"{names} must be device tensors")
    device = first.device
    for t in rest:
        if t is not None:
            if not getattr(t, "is_cuda", False):
                raise TypeError(f"{names} must be device tensors")
            if t.device != device:
                raise ValueError(f"{names} must be on one device")
    return device


def pitch(t, what, align=1):
    """Row pitch of a 2-D tensor whose rows are contiguous: its stride, or (a
    single row, whose stride says nothing) the row's length rounded up."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{what} must be row-major (contiguous rows)")
    if rows > 1:
        return t.stride(0)
    return -(-max(cols, 1) // align) * align


@takes_stream
def quantize_i8(x, out=None, scale=None):
    """Rows of x (float32, float16 or bfloat16) to int8 with one scale each:
    ``scale[i] = max|x[i]| / 127``, ``q[i] = round(x[i] / scale[i])``.

    Returns (q, scale).  A new q has rows of a pitch of 16 bytes, so it can go
    to ``matmul`` and ``matmul_grouped`` whatever its width; its padding is
    not written.  A row of zeros has scale 0; a row with an infinity or NaN
    has that as its scale and zeros.
    """
    import torch
    device = one_device("x, out and scale", x, out, scale)
    if x.dim() != 2:
        raise ValueError("x must have two dimensions")
    code = type_code(x.dtype)
    rows, K = x.shape
    if out is None:
        ldq = -(-K // 16) * 16
        out = torch.empty((rows, ldq), dtype=torch.int8, device=device)
        if ldq != K:
            out = out[:, :K]
    elif out.dtype != torch.int8 or out.shape != x.shape:
        raise ValueError("out must be an int8 tensor of x's shape")
    else:
        ldq = pitch(out, "out")
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=device)
    elif scale.dtype != torch.float32 or scale.shape != (rows,) or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 tensor with one value a row")
    ldx = pitch(x, "x")
    call("quantize_i8", device, rows, K, x.data_ptr(), ldx, code, out.data_ptr(), ldq, scale.data_ptr())
    return out, scale


def gemm_i8(layout, M, N, K, A, lda, B, ldb, C, ldc, scale_a, scale_b, stream=None):
    """Tensor-level int8 call: A, B hold int8 values, C storage of the output
    type (float32, float16 or bfloat16, which its dtype says), scale_a /
    scale_b contiguous float32 tensors of 1 or M / 1 or N values."""
    from .binding import _LAYOUTS, _check_extents
    device = one_device("A, B, C and the scale factors", A, B, C, scale_a, scale_b)
    if A.element_size() != 1 or B.element_size() != 1:
        raise TypeError("int8 operands need 1-byte elements")
    code = type_code(C.dtype)
    _factor_vector(scale_a, M, "scale_a")
    _factor_vector(scale_b, N, "scale_b")
    _check_extents(layout, M, N, K, A, lda, B, ldb, C, ldc, 1, C.element_size())
    lay = _LAYOUTS.get(layout, layout) if isinstance(layout, str) else layout
    run = takes_stream(lambda _, *args: call("gemm_i8_scaled", device, *args))
    run(A, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb, C.data_ptr(), ldc, code,
        scale_a.data_ptr(), scale_a.numel(), scale_b.data_ptr(), scale_b.numel(), lay, stream=stream)


@takes_stream
def matmul_i8(a, b, scale_a, scale_b, out=None, out_dtype=None):
    """``binding.matmul`` for int8 operands: C = (A x B) * scale_a * scale_b,
    the layout read from b's strides as there."""
    import torch
    if scale_a is None or scale_b is None:
        raise ValueError("int8 operands need scale_a and scale_b")
    device = one_device("a, b, out and the scale factors", a, b, out, scale_a, scale_b)
    if b.dtype != torch.int8:
        raise TypeError("a and b must share a dtype")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[0]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} do not chain")
    M, K = a.shape
    N = b.shape[1]
    lda = pitch(a, "a", 16)
    # (A vector as K x 1, strides (1, 1): a column contiguous along K.)
    if b.stride(1) == 1 and (b.stride(0) != 1 or (N == 1 and K <= 1)):
        layout, ldb = 0, (b.stride(0) if K > 1 else -(-max(N, 1) // 16) * 16)
    elif b.stride(0) == 1 or K == 1:
        layout, ldb = 1, (b.stride(1) if N > 1 else -(-max(K, 1) // 16) * 16)
    else:
        raise ValueError("b must be row-major or column-major")
    odt = out_dtype or (out.dtype if out is not None else torch.float32)
    code = type_code(odt)
    if out is None:
        # (One allocation: .t() of a new tensor, and of out for its pitch, cost 1 us each.)
        ldc = max(N if layout == 0 else M, 1)
        out = torch.empty_strided((M, N), (ldc, 1) if layout == 0 else (1, ldc), dtype=odt, device=device)
    elif out.shape != (M, N) or out.dtype != odt:
        raise ValueError("out must be a device tensor of shape (M, N) and the output dtype")
    else:
        ldc = pitch(out if layout == 0 else out.t(), "out (NN) or its transpose (TN)")
    _factor_vector(scale_a, M, "scale_a")
    _factor_vector(scale_b, N, "scale_b")
    if M > 0 and N > 0 and K > 0:
        _need(a, M * lda, "a")
        _need(b, (K if layout == 0 else N) * ldb, "b")
    call("gemm_i8_scaled", device, M, N, K, a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldc, code,
         scale_a.data_ptr(), scale_a.numel(), scale_b.data_ptr(), scale_b.numel(), layout)
    return out


@takes_stream
def matmul_grouped(a, b, offsets, scale_a, scale_b, out=None, out_dtype=None, row_index=None):
    """The int8 products of a mixture of experts over tokens sorted by expert:
    ``out[n] = (a[r] @ b[e].T) * (scale_a[r] * scale_b[e])`` for the rows n of
    expert e, ``offsets[e] <= n < offsets[e + 1]``, with r = n, or
    r = row_index[n].

    a: int8, rows x K; b: int8, experts x N x K (a linear layer's weights, K
    contiguous; both with pitches of a multiple of 16).  offsets: int32,
    experts + 1 values (``expert_sort``).  scale_a: 1 or a's rows values,
    scale_b: 1 or experts x N.  row_index: int32, one row of a for each row of
    the result (its ``token``).  The result has row_index's or a's number of
    rows, float32 unless ``out`` or ``out_dtype`` (float16, bfloat16) says
    otherwise; rows of no expert are not written.
    """
    import torch
    device = one_device("a, b, offsets, row_index, out and the scale factors", a, b, offsets, scale_a, scale_b,
                        row_index, out)
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        raise TypeError("a and b must be int8")
    if a.dim() != 2 or b.dim() != 3 or a.shape[1] != b.shape[2]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} do not chain")
    rows_a, K = a.shape
    G, N = b.shape[:2]
    rows = rows_a
    if row_index is not None:
        if row_index.dtype != torch.int32 or row_index.dim() != 1 or not row_index.is_contiguous():
            raise TypeError("row_index must be a contiguous int32 vector")
        rows = row_index.shape[0]
    if offsets.dtype != torch.int32 or offsets.shape != (G + 1,) or not offsets.is_contiguous():
        raise TypeError("offsets must be a contiguous int32 vector of experts + 1 values")
    _factor_vector(scale_a, rows_a, "scale_a")
    _factor_vector(scale_b, G * N, "scale_b")
    if K > 1 and b.stride(2) != 1:
        raise ValueError("b must be contiguous along K")
    ldb = b.stride(1) if N > 1 else -(-max(K, 1) // 16) * 16
    group_b = b.stride(0) if G > 1 else 0
    lda = pitch(a, "a", 16)
    odt = out_dtype or (out.dtype if out is not None else torch.float32)
    code = type_code(odt)
    if out is None:
        out = torch.empty((rows, N), dtype=odt, device=device)
    if out.shape != (rows, N) or out.dtype != odt:
        raise ValueError("out must be a device tensor with one row for each sorted row, N wide, of the output dtype")
    ldc = pitch(out, "out")
    if rows > 0 and N > 0 and K > 0 and G > 0:
        _need(a, rows_a * lda, "a")
        _need(b, (G - 1) * group_b + N * ldb, "b")
    call("gemm_i8_grouped", device, G, rows, N, K, a.data_ptr(), rows_a, lda,
         row_index.data_ptr() if row_index is not None else None, b.data_ptr(), ldb, group_b, out.data_ptr(), ldc,
         code, scale_a.data_ptr(), scale_a.numel(), scale_b.data_ptr(), scale_b.numel(), offsets.data_ptr())
    return out
