"""Binding of the 8-bit integer linears and of their products grouped by expert
(``include/sketch_int8.h``).

Argument marshalling only, as in the rest of the package: ``sketch_int8_layout``,
``sketch_int8_encode``, ``sketch_int8_swiglu``, ``sketch_int8_workspace_bytes``,
``sketch_int8_matmul``, ``sketch_int8_group_workspace_bytes`` and
``sketch_int8_matmul_group`` have the names of the C ABI; the rest is a
convenience layer over them.
"""
import ctypes
import functools

import torch

from . import OK, SketchError, _check, _ptr, _stream_handle, dtype_code, lib, sketch_encode_status
from .fp8 import _aligned, _given, _need, _On, _out, _remember, _shared

INT8_ROWS = 4               # x_dtype of rows that an encoder wrote
INT8_TOKENS = 16            # rows that a product may encode as it reads them
INT8_MAX_N, INT8_MAX_M, INT8_MAX_EXPERTS = 131071, 1 << 24, 512
INT8_EXPORTS = ("sketch_int8_layout", "sketch_int8_encode", "sketch_int8_swiglu", "sketch_int8_workspace_bytes",
                "sketch_int8_matmul", "sketch_int8_group_workspace_bytes", "sketch_int8_matmul_group")


class Int8Params(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("count", ctypes.c_int32)]


class Int8Shape(ctypes.Structure):
    _fields_ = [("ld", ctypes.c_int64), ("scales_offset", ctypes.c_size_t), ("bytes", ctypes.c_size_t)]


class Int8Groups(ctypes.Structure):
    _fields_ = [("terms", ctypes.c_int64), ("counts", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("counts_bits", ctypes.c_int32), ("rows_bits", ctypes.c_int32)]


_declared = None


def _int8_lib():
    global _declared
    if _declared is None:
        L = lib()
        P, G = ctypes.POINTER(Int8Params), ctypes.POINTER(Int8Groups)
        vp, i64, sz, it = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        L.sketch_int8_layout.argtypes = [P, ctypes.POINTER(Int8Shape)]
        L.sketch_int8_encode.argtypes = [P, vp, it, i64, vp, vp, vp]
        L.sketch_int8_swiglu.argtypes = [P, vp, i64, vp, i64, it, vp, vp, vp]
        L.sketch_int8_workspace_bytes.argtypes = [P, i64, it, it, ctypes.POINTER(sz)]
        L.sketch_int8_matmul.argtypes = [P, vp, vp, it, i64, vp, it, vp, sz, vp]
        L.sketch_int8_group_workspace_bytes.argtypes = [P, i64, i64, it, it, ctypes.POINTER(sz)]
        L.sketch_int8_matmul_group.argtypes = [P, vp, vp, it, i64, G, vp, it, vp, sz, vp]
        for name in INT8_EXPORTS:
            getattr(L, name).restype = it
        _declared = L
    return _declared


# ---------------------------------------------------------------------------
# thin wrappers of the C ABI (same names)
# ---------------------------------------------------------------------------

def sketch_int8_layout(p):
    s = Int8Shape()
    _check(_int8_lib().sketch_int8_layout(ctypes.byref(p), ctypes.byref(s)), "sketch_int8_layout")
    return s


def sketch_int8_encode(p, W, ldw, buf, status=None, stream=None):
    """status: an int32 device tensor the kernel ORs flags into, or None."""
    stream = stream if stream is not None else _stream_handle(W.device)
    _check(_int8_lib().sketch_int8_encode(ctypes.byref(p), _ptr(W), dtype_code(W), int(ldw), _ptr(buf), _ptr(status),
                                          stream), "sketch_int8_encode")


def sketch_int8_swiglu(p, gate, ld_gate, up, ld_up, buf, status=None, stream=None):
    stream = stream if stream is not None else _stream_handle(gate.device)
    _check(_int8_lib().sketch_int8_swiglu(ctypes.byref(p), _ptr(gate), int(ld_gate), _ptr(up), int(ld_up),
                                          dtype_code(gate), _ptr(buf), _ptr(status), stream), "sketch_int8_swiglu")


def sketch_int8_workspace_bytes(p, batch, x_dtype, y_dtype):
    n = ctypes.c_size_t()
    _check(_int8_lib().sketch_int8_workspace_bytes(ctypes.byref(p), int(batch), int(x_dtype), int(y_dtype),
                                                   ctypes.byref(n)), "sketch_int8_workspace_bytes")
    return n.value


def sketch_int8_matmul(p, buf, X, x_dtype, batch, Y, workspace, stream=None):
    stream = stream if stream is not None else _stream_handle(Y.device)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_int8_lib().sketch_int8_matmul(ctypes.byref(p), _ptr(buf), _ptr(X), int(x_dtype), int(batch), _ptr(Y),
                                          dtype_code(Y), _ptr(workspace), wsb, stream), "sketch_int8_matmul")


def sketch_int8_group_workspace_bytes(p, terms, x_rows, x_dtype, y_dtype):
    n = ctypes.c_size_t()
    _check(_int8_lib().sketch_int8_group_workspace_bytes(ctypes.byref(p), int(terms), int(x_rows), int(x_dtype),
                                                         int(y_dtype), ctypes.byref(n)),
           "sketch_int8_group_workspace_bytes")
    return n.value


def sketch_int8_matmul_group(p, buf, X, x_dtype, x_rows, groups, Y, workspace, stream=None):
    stream = stream if stream is not None else _stream_handle(Y.device)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_int8_lib().sketch_int8_matmul_group(ctypes.byref(p), _ptr(buf), _ptr(X), int(x_dtype), int(x_rows),
                                                ctypes.byref(groups), _ptr(Y), dtype_code(Y), _ptr(workspace), wsb,
                                                stream), "sketch_int8_matmul_group")


# ---------------------------------------------------------------------------
# high-level API
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=1024)
def _shape(M, N, count):
    """Parameters, their reference and the layout of one kind of buffer, shared
    by all of it: never handed out."""
    p = Int8Params(M, N, count)
    return p, ctypes.byref(p), sketch_int8_layout(p)


class Int8Tables:
    """A matrix [M, N] (or a stack [count, M, N]) as int8 codes and a float32
    scale for each row, in the buffer layout of the C ABI (a uint8 device
    tensor).  Its values may be changed, its shape and buffer not: `params` and
    `layout` are copies.  The products read the padding behind a row's N codes,
    which has to be zero: a table made here starts as zeros, the padding of a
    `buf` that is given is the caller's."""

    def __init__(self, M, N, count=None, device="cuda", buf=None, *, _zero=True):
        if count is not None and count < 1:
            raise ValueError("an empty stack of matrices")
        self._M, self._N, self._count = int(M), int(N), None if count is None else int(count)
        self._params, self._ref, self._layout = _shape(self._M, self._N, self._count or 1)
        n = (self._count or 1) * self._layout.bytes
        if buf is None:
            self._codes = (torch.zeros if _zero else torch.empty)(n, dtype=torch.int8, device=device)
        else:
            _need(buf.dtype == torch.uint8 and buf.is_contiguous() and buf.numel() >= n and buf.data_ptr() % 16 == 0,
                  "the buffer must be %d dense, 16-byte aligned bytes" % n)
            self._codes = buf.view(-1).view(torch.int8)
        self._device, self._at = self._codes.device, self._codes.data_ptr()
        self._ws = {}

    M = property(lambda self: self._M)
    N = property(lambda self: self._N)
    count = property(lambda self: self._count)
    device = property(lambda self: self._device)
    buf = property(lambda self: self._codes.view(torch.uint8))
    params = property(lambda self: Int8Params.from_buffer_copy(self._params))
    layout = property(lambda self: Int8Shape.from_buffer_copy(self._layout))

    @property
    def shape(self):
        return ((self._M, self._N) if self._count is None else (self._count, self._M, self._N))

    def codes(self):
        """The codes as an int8 view (rows are padded: not contiguous unless N % 128 == 0)."""
        s, at = self._layout, self._codes.storage_offset()
        if self._count is None:
            return self._codes.as_strided((self._M, self._N), (s.ld, 1), at)
        return self._codes.as_strided((self._count, self._M, self._N), (s.bytes, s.ld, 1), at)

    def scales(self):
        """The scales, float32 [M] (a view)."""
        s = self._layout
        at = self._codes.storage_offset() + s.scales_offset
        if self._count is None:
            return self._codes.as_strided((4 * self._M,), (1,), at).view(torch.float32)
        return self._codes.as_strided((self._count, 4 * self._M), (s.bytes, 1), at).view(torch.float32)


def _rows_of(x):
    """(x, its row stride), or a copy where its rows are not dense and evenly apart."""
    stride = x.stride()
    if len(stride) == 2 and stride[1] == 1 and stride[0] >= x.shape[1]:
        return x, stride[0]
    rows, N = x.shape[-2:]
    dense = N <= 1 or stride[-1] == 1
    even = x.dim() == 2 or x.shape[0] <= 1 or stride[0] == rows * stride[1]
    if dense and x.dim() == 2 and rows <= 1:
        return x, N
    return (x, stride[-2]) if dense and even and stride[-2] >= N else (x.contiguous(), N)


def _flags(status, device):
    if status is not None:
        _need(status.dtype == torch.int32 and status.numel() >= 1 and status.device == device,
              "status must be an int32 tensor on the same device")


def int8_encode(W, check=True, status=None):
    """Encode W [M, N], or a stack [count, M, N] of matrices, float32, bfloat16
    or float16 on a GPU, row by row: weights by output channel, activations by
    token.

    With check=True the call waits for the device and raises SketchError when
    an element is NaN or infinite; with check=False it stays asynchronous (such
    a row has the scale NaN) and ORs flags into `status`, a zeroed int32 device
    tensor of one element, when given."""
    if W.dim() not in (2, 3) or not W.is_cuda:
        raise ValueError("W must be a 2-D GPU tensor, or a 3-D one for a stack of matrices")
    _flags(status, W.device)
    dtype = dtype_code(W)
    W, ld = _rows_of(W)
    t = Int8Tables(W.shape[-2], W.shape[-1], W.shape[0] if W.dim() == 3 else None, W.device, _zero=False)
    with _On(W.device) as stream:
        if check and status is None:
            status = torch.zeros(1, dtype=torch.int32, device=W.device)
        rc = _int8_lib().sketch_int8_encode(t._ref, W.data_ptr(), dtype, ld, t._at,
                                            status.data_ptr() if status is not None else None, stream)
        if rc != OK:
            raise SketchError(rc, "sketch_int8_encode")
        if check:
            flags = int(status.item())
            rc = sketch_encode_status(flags)
            if rc != OK:
                raise SketchError(rc, "sketch_int8_encode (device flags 0x%x)" % flags)
    return t


def int8_swiglu(gate, up, status=None):
    """Int8Tables of the rows of silu(gate) * up, gate and up [T, N] of one type
    (views with a row stride, such as the halves of one product's rows, are read
    in place): the activations between the products of an MLP.  Asynchronous; a
    row with a value that is NaN or infinite has the scale NaN, and ORs a flag
    into `status`, an int32 device tensor, when given."""
    shape, device = gate.shape, gate.device
    if len(shape) != 2 or not gate.is_cuda or shape != up.shape:
        raise ValueError("gate and up must be 2-D GPU tensors of one shape")
    if gate.dtype != up.dtype or device != up.device:
        raise ValueError("gate and up must have one dtype and device")
    _flags(status, device)
    dtype = dtype_code(gate)
    gate, ld_gate = _rows_of(gate)
    up, ld_up = _rows_of(up)
    t = Int8Tables(*shape, None, device, _zero=False)
    with _On(device) as stream:
        rc = _int8_lib().sketch_int8_swiglu(t._ref, gate.data_ptr(), ld_gate, up.data_ptr(), ld_up, dtype, t._at,
                                            status.data_ptr() if status is not None else None, stream)
    if rc != OK:
        raise SketchError(rc, "sketch_int8_swiglu")
    return t


def int8_tables(codes, scales):
    """Int8Tables from codes [M, N] (int8) and scales [M] (float32), or stacks of
    both: a copy into the library's layout."""
    _need(codes.dtype == torch.int8 and scales.dtype == torch.float32, "codes must be int8 and scales float32")
    _need(codes.dim() in (2, 3) and codes.is_cuda and scales.device == codes.device,
          "codes and scales must be tensors on one GPU, codes 2-D (or 3-D)")
    _need(scales.shape == codes.shape[:-1], "scales must have shape %s" % (tuple(codes.shape[:-1]),))
    t = Int8Tables(codes.shape[-2], codes.shape[-1], codes.shape[0] if codes.dim() == 3 else None, codes.device)
    t.codes().copy_(codes)
    t.scales().copy_(scales)
    return t


def _workspace_bytes(t, batch, x_dtype, y_dtype):
    key = (batch, x_dtype, y_dtype)
    n = t._ws.get(key)
    if n is None:
        n = _remember(t._ws, key, sketch_int8_workspace_bytes(t._params, batch, x_dtype, y_dtype))
    return n


def _group_workspace_bytes(t, terms, x_rows, x_dtype, y_dtype):
    key = (terms, x_rows, x_dtype, y_dtype)
    n = t._ws.get(key)
    if n is None:
        n = _remember(t._ws, key, sketch_int8_group_workspace_bytes(t._params, terms, x_rows, x_dtype, y_dtype))
    return n


def int8_workspace_for(t, batch, x_dtype, y_dtype, device):
    """Workspace for products of `batch` rows (None if not needed).  Reuse it
    across calls on one stream, never for two calls in flight at once."""
    with _On(t.device):
        n = _workspace_bytes(t, batch, x_dtype, y_dtype)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def int8_group_workspace_for(t, terms, x_rows, x_dtype, y_dtype, device):
    """The same for products grouped by expert: `terms` rows of Y, `x_rows` of X."""
    with _On(t.device):
        n = _group_workspace_bytes(t, terms, x_rows, x_dtype, y_dtype)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _operand(t, X):
    """(x_dtype, the tensor or tables that hold it) of X, checked against the weight t."""
    if isinstance(X, Int8Tables):
        _need(X._count is None, "encoded rows must be one matrix")
        x, xdt = X, INT8_ROWS
    else:
        xdt, x = dtype_code(X), _aligned(X)
    if X.device != t._device:
        raise ValueError("X and the weight are on different devices")
    return xdt, x


def int8_matmul(t, X, out=None, workspace=None, dtype=None):
    """Y = X8 . W8^T [batch, M] for an encoded weight t and X [batch, N] (or
    [N]), encoded row by row on the way in; X may also be the Int8Tables of
    encoded rows, which several linears can share.  dtype: of Y, float32 (the
    default, or that of `out`), bfloat16 or float16.  The sums are exact.  `out`
    may share memory with X (of up to INT8_TOKENS rows a copy is made), not with
    the weight or with encoded rows."""
    if t._count is not None:
        raise ValueError("t must be one weight")
    shape = X.shape
    if len(shape) not in (1, 2) or shape[-1] != t._N:
        raise ValueError("X must have %d columns, got shape %s" % (t._N, tuple(shape)))
    squeeze = len(shape) == 1
    batch = 1 if squeeze else shape[0]
    xdt, x = _operand(t, X)
    device = t._device
    if xdt == INT8_ROWS:
        at = x._at
    else:
        if out is not None and batch <= INT8_TOKENS and _shared(x, out):
            x = x.clone()
        at = x.data_ptr()
    shape = (t._M,) if squeeze else (batch, t._M)
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    with _On(device) as stream:
        Y = torch.empty(shape, dtype=dtype, device=device) if out is None else _out(out, shape, dtype, device)
        ydt = dtype_code(Y)
        if workspace is None:
            wsb = _workspace_bytes(t, batch, xdt, ydt)
            workspace = torch.empty(wsb, dtype=torch.uint8, device=device) if wsb else None
        else:
            wsb = _given(workspace, device)
        rc = _int8_lib().sketch_int8_matmul(t._ref, t._at, at, xdt, batch, Y.data_ptr(), ydt,
                                            workspace.data_ptr() if workspace is not None else None, wsb, stream)
    if rc != OK:
        raise SketchError(rc, "sketch_int8_matmul")
    return Y


def _integers(x, name, n, device):
    """A dense int32 or int64 vector, and its bits."""
    _need(x.dtype in (torch.int32, torch.int64) and x.dim() == 1 and x.device == device and (n is None or x.shape[0] == n),
          "%s must be an int32 or int64 vector%s on the weights' device" % (name, "" if n is None else " of %d" % n))
    return x.contiguous(), 32 if x.dtype == torch.int32 else 64


def int8_matmul_group(t, X, counts, rows=None, out=None, workspace=None, dtype=None):
    """Products grouped by expert: Y [terms, M] for a stack t of E encoded
    weights [E, M, N].  The terms, pairs of a row of X and an expert, stand in
    the order of their experts, counts[e] of them for expert e (int32 or int64
    [E] on the device: nothing waits for the host).  Term i takes row rows[i] of
    X [x_rows, N] (int32 or int64 [terms]; a row outside X gives NaN), or row i
    without `rows`.  X is encoded row by row on the way in, or is the Int8Tables
    of encoded rows.  dtype: of Y, float32 (the default, or that
    of `out`), bfloat16 or float16.  Rows of Y behind the last term are left as
    they were (an `out` that is not given holds anything there).  `out` may share
    memory with X (a copy is made), not with the weights or with encoded rows."""
    if t._count is None:
        raise ValueError("t must be a stack of weights")
    shape, device = X.shape, t._device
    if len(shape) != 2 or shape[1] != t._N:
        raise ValueError("X must be [rows, %d], got shape %s" % (t._N, tuple(shape)))
    xdt, x = _operand(t, X)
    counts, counts_bits = _integers(counts, "counts", t._count, device)
    rows_at, rows_bits, terms = None, 0, shape[0]
    if rows is not None:
        rows, rows_bits = _integers(rows, "rows", None, device)
        rows_at, terms = rows.data_ptr(), rows.shape[0]
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    with _On(device) as stream:
        Y = torch.empty((terms, t._M), dtype=dtype, device=device) if out is None else \
            _out(out, (terms, t._M), dtype, device)
        ydt = dtype_code(Y)
        if xdt != INT8_ROWS and out is not None and _shared(x, out):
            x = x.clone()
        if workspace is None:
            wsb = _group_workspace_bytes(t, terms, shape[0], xdt, ydt)
            workspace = torch.empty(wsb, dtype=torch.uint8, device=device) if wsb else None
        else:
            wsb = _given(workspace, device)
        groups = Int8Groups(terms, counts.data_ptr(), rows_at, counts_bits, rows_bits)
        rc = _int8_lib().sketch_int8_matmul_group(
            t._ref, t._at, x._at if xdt == INT8_ROWS else x.data_ptr(), xdt, shape[0], ctypes.byref(groups),
            Y.data_ptr(), ydt, workspace.data_ptr() if workspace is not None else None, wsb, stream)
    if rc != OK:
        raise SketchError(rc, "sketch_int8_matmul_group")
    return Y
