"""Binding of the 8-bit floating-point linears and of the mixture-of-experts
layer (``include/sketch_fp8.h``).

Argument marshalling only, as in the rest of the package: ``sketch_fp8_layout``,
``sketch_fp8_encode``, ``sketch_fp8_workspace_bytes``, ``sketch_fp8_matmul``,
``sketch_moe_workspace_bytes`` and ``sketch_moe`` have the names of the C ABI;
the rest is a convenience layer over them.
"""
import ctypes
import functools

import torch

from . import BF16, OK, SketchError, _check, _ptr, _stream_handle, dtype_code, lib, sketch_encode_status

FP8_ROWS = 3                # x_dtype of rows that sketch_fp8_encode wrote
FP8_F32_SUMS = 256          # with y_dtype BF16: float32 sums for any number of rows
FP8_EXACT_BATCH = 64        # rows up to which a bfloat16 Y has them anyway
FP8_TOKENS = 4              # rows that a product encodes as it reads them
MOE_MAX_EXPERTS, MOE_MAX_TOPK, MOE_MAX_TOKENS = 512, 16, 64
FP8_EXPORTS = ("sketch_fp8_layout", "sketch_fp8_encode", "sketch_fp8_workspace_bytes", "sketch_fp8_matmul",
               "sketch_moe_workspace_bytes", "sketch_moe")


class Fp8Params(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("block_rows", ctypes.c_int32),
                ("count", ctypes.c_int32)]


class Fp8Shape(ctypes.Structure):
    _fields_ = [("ld", ctypes.c_int64), ("row_blocks", ctypes.c_int64), ("col_blocks", ctypes.c_int64),
                ("lds", ctypes.c_int64), ("scales_offset", ctypes.c_size_t), ("bytes", ctypes.c_size_t)]


class MoEParams(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("x_dtype", ctypes.c_int)]


_declared = None


def _fp8_lib():
    global _declared
    if _declared is None:
        L = lib()
        P, Q = ctypes.POINTER(Fp8Params), ctypes.POINTER(MoEParams)
        vp, i64, sz, it = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        L.sketch_fp8_layout.argtypes = [P, ctypes.POINTER(Fp8Shape)]
        L.sketch_fp8_encode.argtypes = [P, vp, it, vp, vp, vp]
        L.sketch_fp8_workspace_bytes.argtypes = [P, i64, it, it, ctypes.POINTER(sz)]
        L.sketch_fp8_matmul.argtypes = [P, vp, vp, it, i64, vp, it, vp, sz, vp]
        L.sketch_moe_workspace_bytes.argtypes = [Q, i64, ctypes.POINTER(sz)]
        L.sketch_moe.argtypes = [Q, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, sz, vp]
        for name in FP8_EXPORTS:
            getattr(L, name).restype = it
        _declared = L
    return _declared


# ---------------------------------------------------------------------------
# thin wrappers of the C ABI (same names)
# ---------------------------------------------------------------------------

def sketch_fp8_layout(p):
    s = Fp8Shape()
    _check(_fp8_lib().sketch_fp8_layout(ctypes.byref(p), ctypes.byref(s)), "sketch_fp8_layout")
    return s


def sketch_fp8_encode(p, W, buf, status=None, stream=None):
    """status: an int32 device tensor the kernel ORs flags into, or None."""
    stream = stream if stream is not None else _stream_handle(W.device)
    _check(_fp8_lib().sketch_fp8_encode(ctypes.byref(p), _ptr(W), dtype_code(W), _ptr(buf), _ptr(status), stream),
           "sketch_fp8_encode")


def _y_dtype(Y, float32_sums):
    code = dtype_code(Y)
    return code | FP8_F32_SUMS if float32_sums and code == BF16 else code


def sketch_fp8_workspace_bytes(p, batch, x_dtype, y_dtype):
    n = ctypes.c_size_t()
    _check(_fp8_lib().sketch_fp8_workspace_bytes(ctypes.byref(p), int(batch), int(x_dtype), int(y_dtype),
                                                 ctypes.byref(n)), "sketch_fp8_workspace_bytes")
    return n.value


def sketch_fp8_matmul(p, buf, X, x_dtype, batch, Y, workspace, stream=None, float32_sums=False):
    stream = stream if stream is not None else _stream_handle(Y.device)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_fp8_lib().sketch_fp8_matmul(ctypes.byref(p), _ptr(buf), _ptr(X), int(x_dtype), int(batch), _ptr(Y),
                                        _y_dtype(Y, float32_sums), _ptr(workspace), wsb, stream), "sketch_fp8_matmul")


def sketch_moe_workspace_bytes(p, tokens):
    n = ctypes.c_size_t()
    _check(_fp8_lib().sketch_moe_workspace_bytes(ctypes.byref(p), int(tokens), ctypes.byref(n)),
           "sketch_moe_workspace_bytes")
    return n.value


def sketch_moe(p, router, gate, up, down, X, Y, ids, weights, workspace, stream=None):
    stream = stream if stream is not None else _stream_handle(X.device)
    wsb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_fp8_lib().sketch_moe(ctypes.byref(p), _ptr(router), _ptr(gate), _ptr(up), _ptr(down), _ptr(X), X.shape[0],
                                 _ptr(Y), _ptr(ids), _ptr(weights), _ptr(workspace), wsb, stream), "sketch_moe")


# ---------------------------------------------------------------------------
# high-level API
# ---------------------------------------------------------------------------

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device   # a tensor on the GPU exists


class _On:
    """The device made current for the call, if it is not (launches go to the
    current device); `with` gives the current stream of the device."""

    def __init__(self, device):
        self.index, self.other = device.index, None

    def __enter__(self):
        if self.index is None:
            raise ValueError("tensors must be on a GPU")
        if _current_device() != self.index:
            self.other = torch.cuda.device(self.index)
            self.other.__enter__()
        return _raw_stream(self.index)

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _aligned(t):
    """t itself when dense and 16-byte aligned, else a copy that is."""
    if not t.is_contiguous():
        return t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


@functools.lru_cache(maxsize=1024)
def _shape(M, N, block_rows, count):
    """Parameters, their reference and the layout of one kind of buffer, shared
    by all of it: never handed out."""
    p = Fp8Params(M, N, block_rows, count)
    return p, ctypes.byref(p), sketch_fp8_layout(p)


class Fp8Tables:
    """A matrix [M, N] (or a stack [count, M, N]) as e4m3 codes and block
    scales, in the buffer layout of the C ABI (a uint8 device tensor).  Its
    values may be changed, its shape and buffer not: `params` and `layout` are
    copies.  The products read the padding behind a row's codes and scales, which
    has to be zero: a table made here starts as zeros, the padding of a `buf` that
    is given is the caller's."""

    def __init__(self, M, N, block_rows=128, count=None, device="cuda", buf=None, *, _zero=True):
        if count is not None and count < 1:
            raise ValueError("an empty stack of matrices")
        stack = 1 if count is None else int(count)
        self._M, self._N, self._block_rows, self._count = int(M), int(N), int(block_rows), None if count is None else stack
        self._params, self._ref, self._layout = _shape(self._M, self._N, self._block_rows, stack)
        n = stack * self._layout.bytes
        if buf is None:
            buf = (torch.zeros if _zero else torch.empty)(n, dtype=torch.uint8, device=device)
        else:
            _need(buf.dtype == torch.uint8 and buf.is_contiguous() and buf.numel() >= n and buf.data_ptr() % 16 == 0,
                  "the buffer must be %d dense, 16-byte aligned bytes" % n)
        self._buf, self._device, self._at = buf, buf.device, buf.data_ptr()
        self._ws = {}

    M = property(lambda self: self._M)
    N = property(lambda self: self._N)
    block_rows = property(lambda self: self._block_rows)
    count = property(lambda self: self._count)
    device = property(lambda self: self._device)
    buf = property(lambda self: self._buf)
    params = property(lambda self: Fp8Params.from_buffer_copy(self._params))
    layout = property(lambda self: Fp8Shape.from_buffer_copy(self._layout))

    @property
    def shape(self):
        return ((self.M, self.N) if self.count is None else (self.count, self.M, self.N))

    def _view(self, rows, cols, ld, at):
        if self.count is None:
            return self._buf.as_strided((rows, cols), (ld, 1), self._buf.storage_offset() + at)
        return self._buf.as_strided((self._count, rows, cols), (self._layout.bytes, ld, 1), self._buf.storage_offset() + at)

    def codes(self):
        """The codes as a float8_e4m3fn view (rows are padded: not contiguous unless N % 128 == 0)."""
        return self._view(self._M, self._N, self._layout.ld, 0).view(torch.float8_e4m3fn)

    def scales(self):
        """The biased scale exponents, uint8 [row blocks, column blocks] (a view): scale = 2^(byte - 127)."""
        s = self._layout
        return self._view(s.row_blocks, s.col_blocks, s.lds, s.scales_offset)


def fp8_encode(W, block_rows=128, check=True, status=None):
    """Encode W [M, N], or a stack [count, M, N] of matrices, float32,
    bfloat16 or float16 on a GPU, in blocks of 128 x 128 (weights) or, with
    block_rows=1, of 1 x 128 (activations).

    With check=True the call waits for the device and raises SketchError when
    an element is NaN or infinite; with check=False it stays asynchronous (such
    a block encodes to NaN) and ORs flags into `status`, a zeroed int32 device
    tensor of one element, when given."""
    if W.dim() not in (2, 3) or not W.is_cuda:
        raise ValueError("W must be a 2-D GPU tensor, or a 3-D one for a stack of matrices")
    if status is not None:
        _need(status.dtype == torch.int32 and status.numel() >= 1 and status.device == W.device,
              "status must be an int32 tensor on W's device")
    dtype_code(W)
    W = _aligned(W)
    t = Fp8Tables(W.shape[-2], W.shape[-1], block_rows, W.shape[0] if W.dim() == 3 else None, W.device,
                  _zero=False)
    with _On(W.device) as stream:
        if check and status is None:
            status = torch.zeros(1, dtype=torch.int32, device=W.device)
        sketch_fp8_encode(t._params, W, t.buf, status, stream)
        if check:
            flags = int(status.item())
            rc = sketch_encode_status(flags)
            if rc != OK:
                raise SketchError(rc, "sketch_fp8_encode (device flags 0x%x)" % flags)
    return t


def fp8_tables(codes, scales, block_rows=128):
    """Fp8Tables from codes [M, N] (float8_e4m3fn, or their uint8 bits) and
    biased scale exponents [row blocks, column blocks] (float8_e8m0fnu, or
    uint8), or stacks of both: a copy into the library's layout."""
    _need(codes.dtype in (torch.uint8, torch.float8_e4m3fn) and scales.dtype in (torch.uint8, torch.float8_e8m0fnu),
          "codes must be float8_e4m3fn and scales float8_e8m0fnu, or the uint8 bits of these")
    codes, scales = codes.view(torch.uint8), scales.view(torch.uint8)
    _need(codes.dim() in (2, 3) and codes.is_cuda and scales.device == codes.device,
          "codes and scales must be 2-D (or 3-D) tensors on one GPU")
    count = codes.shape[0] if codes.dim() == 3 else None
    t = Fp8Tables(codes.shape[-2], codes.shape[-1], block_rows, count, codes.device)
    want = (t._layout.row_blocks, t._layout.col_blocks)
    _need(tuple(scales.shape) == (want if count is None else (count,) + want), "scales must have shape %s" % (want,))
    t._view(t.M, t.N, t._layout.ld, 0).copy_(codes)
    t.scales().copy_(scales)
    return t


_SIZES = 1024               # workspace sizes that a table remembers


def _remember(sizes, key, n):
    """n, kept in `sizes`, which starts anew once it is full: a program meets any
    number of batch sizes as it runs."""
    if len(sizes) >= _SIZES:
        sizes.clear()
    sizes[key] = n
    return n


def _workspace_bytes(t, batch, x_dtype, y_dtype):
    key = (batch, x_dtype, y_dtype)
    n = t._ws.get(key)
    if n is None:
        n = _remember(t._ws, key, sketch_fp8_workspace_bytes(t._params, batch, x_dtype, y_dtype))
    return n


def fp8_workspace_for(t, batch, x_dtype, y_dtype, device):
    """Workspace for products of `batch` rows (None if not needed).  Reuse it
    across calls on one stream, never for two calls in flight at once.  y_dtype:
    the code of Y's type, BF16 | FP8_F32_SUMS for float32_sums."""
    with _On(t.device):
        n = _workspace_bytes(t, batch, x_dtype, y_dtype)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _given(workspace, device):
    """Bytes of a workspace the caller gave."""
    _need(workspace.device == device and workspace.is_contiguous(), "the workspace must be dense, on the same device")
    return workspace.numel() * workspace.element_size()


def _out(out, shape, dtype, device):
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(tuple(out.shape) == tuple(shape) and out.dtype == dtype and out.is_contiguous() and out.device == device,
          "out must be a dense %s tensor %s on the same device" % (dtype, tuple(shape)))
    return out


def _shared(a, b):
    """Whether two dense tensors have bytes in common."""
    p, q = a.data_ptr(), b.data_ptr()
    return p < q + b.numel() * b.element_size() and q < p + a.numel() * a.element_size()


def fp8_matmul(t, X, out=None, workspace=None, dtype=None, float32_sums=False):
    """Y = X8 . W8^T [batch, M] for an encoded weight t and X [batch, N] (or
    [N]), encoded row by row on the way in; X may also be an Fp8Tables with
    block_rows=1, for rows that several linears share.  dtype: of Y, float32
    (the default, or that of `out`), bfloat16 or float16.  Sums are float32, but
    for a bfloat16 Y of more than FP8_EXACT_BATCH rows, which is summed on the
    e4m3 matrix cores (twice as fast; include/sketch_fp8.h states the error)
    unless float32_sums is true.  `out` may share memory with X (of up to
    FP8_TOKENS rows a copy is made), not with the weight or with encoded rows."""
    if t._block_rows != 128 or t._count is not None:
        raise ValueError("t must be one weight, encoded with block_rows=128")
    rows = isinstance(X, Fp8Tables)
    if rows:
        _need(X.block_rows == 1 and X.count is None, "encoded rows must have block_rows=1")
    shape, device = X.shape, t._device
    if X.device != device:
        raise ValueError("X and the weight are on different devices")
    if len(shape) not in (1, 2) or shape[-1] != t._N:
        raise ValueError("X must have %d columns, got shape %s" % (t._N, tuple(shape)))
    squeeze = len(shape) == 1
    batch = 1 if squeeze else shape[0]
    if rows:
        xdt, at = FP8_ROWS, X._at
    else:
        xdt, x = dtype_code(X), _aligned(X)
        if out is not None and batch <= FP8_TOKENS and _shared(x, out):
            x = x.clone()
        at = x.data_ptr()
    shape = (t._M,) if squeeze else (batch, t._M)
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    with _On(device) as stream:
        Y = torch.empty(shape, dtype=dtype, device=device) if out is None else _out(out, shape, dtype, device)
        ydt = _y_dtype(Y, float32_sums)
        if workspace is None:
            wsb = _workspace_bytes(t, batch, xdt, ydt)
            workspace = torch.empty(wsb, dtype=torch.uint8, device=device) if wsb else None
        else:
            wsb = _given(workspace, device)
        rc = _fp8_lib().sketch_fp8_matmul(t._ref, t._at, at, xdt, batch, Y.data_ptr(), ydt,
                                          workspace.data_ptr() if workspace is not None else None, wsb, stream)
    if rc != OK:
        raise SketchError(rc, "sketch_fp8_matmul")
    return Y


class MoE:
    """A mixture-of-experts layer: router [E, H] (float32, bfloat16 or
    float16, the dtype its tokens have) and the experts' weights, stacks of E
    encoded matrices: gate and up [E, I, H], down [E, H, I].  renorm: whether
    the weights of the chosen experts are scaled to sum to one.  The layer
    reads these tensors' values at each call (a copy of a router that is not
    dense and 16-byte aligned: layer.router)."""

    def __init__(self, router, gate, up, down, topk, renorm=True):
        _need(router.dim() == 2 and router.is_cuda, "router must be a 2-D GPU tensor")
        E, H = router.shape
        for name, t in (("gate", gate), ("up", up), ("down", down)):
            _need(isinstance(t, Fp8Tables) and t.block_rows == 128 and t.count == E and t.device == router.device,
                  "%s must be a stack of %d weights, encoded with block_rows=128, on the router's device" % (name, E))
        I = gate.M
        _need(gate.shape == up.shape == (E, I, H) and down.shape == (E, H, I),
              "gate and up must be [E, I, H], down [E, H, I], the router [E, H]")
        self._tensors = _aligned(router), gate, up, down
        self._topk, self._renorm = int(topk), bool(renorm)
        self._params = MoEParams(H, I, E, self._topk, int(self._renorm), dtype_code(router))
        self._fixed = (ctypes.byref(self._params), self.router.data_ptr(), gate._at, up._at, down._at)
        self._H, self._dtype, self._device = H, router.dtype, router.device
        sketch_moe_workspace_bytes(self._params, 0)   # checks the sizes
        self._ws = {}

    # a layer's values may be changed in place, its tensors and sizes not (`params` is a copy)
    params = property(lambda self: MoEParams.from_buffer_copy(self._params))
    router = property(lambda self: self._tensors[0])
    gate = property(lambda self: self._tensors[1])
    up = property(lambda self: self._tensors[2])
    down = property(lambda self: self._tensors[3])
    topk = property(lambda self: self._topk)
    renorm = property(lambda self: self._renorm)

    def _workspace_bytes(self, tokens):
        n = self._ws.get(tokens)
        if n is None:
            n = self._ws[tokens] = max(sketch_moe_workspace_bytes(self._params, tokens), 16)
        return n

    def workspace_for(self, tokens):
        """Workspace for `tokens` tokens.  Reuse it across calls on one
        stream, never for two calls in flight at once."""
        with _On(self._device):
            n = self._workspace_bytes(tokens)
        return torch.empty(n, dtype=torch.uint8, device=self._device)


def moe(layer, X, out=None, workspace=None, return_routing=False):
    """Y float32 [tokens, H] of a MoE layer for X [tokens, H] (up to
    MOE_MAX_TOKENS tokens, of the router's dtype); with return_routing also
    the chosen experts int32 [tokens, topk], by descending logit, and their
    weights float32 [tokens, topk].  `out` may share memory with X."""
    shape, dev, k = X.shape, layer._device, layer._topk
    if len(shape) != 2 or shape[1] != layer._H:
        raise ValueError("X must be [tokens, %d]" % layer._H)
    if X.dtype != layer._dtype or X.device != dev:
        raise ValueError("X must have the router's dtype and device")
    X, T = _aligned(X), shape[0]
    with _On(dev) as stream:
        Y = torch.empty(shape, dtype=torch.float32, device=dev) if out is None else _out(out, shape, torch.float32, dev)
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        if workspace is None:
            wsb = layer._workspace_bytes(T)
            workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
        else:
            wsb = _given(workspace, dev)
        rc = _fp8_lib().sketch_moe(*layer._fixed, X.data_ptr(), T, Y.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                                   workspace.data_ptr(), wsb, stream)
    if rc != OK:
        raise SketchError(rc, "sketch_moe")
    return (Y, ids, weights) if return_routing else Y
