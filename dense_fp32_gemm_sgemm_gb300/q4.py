"""4-bit weights: packed matrices, few-row products and the mixture-of-experts layer.

Like the rest of the binding this marshals arguments only; the layout, the arithmetic and
the limits are those of the ``sgemm_q4_*`` and ``sgemm_moe`` entry points in the C header.

    W = sg.q4_quantize(B, group=128)          # B: N x K (or E x N x K), any float type
    C = sg.q4_matmul(A, W)                    # A: M x N, a few rows; C has A's type
    C = sg.matmul(A, sg.q4_dequantize(W))     # many float32 rows, N and K up to 8192
    layer = sg.MoeLayer(router, gate, up, down, top_k=2)
    y, ids, weights = layer(x)                # x: T x D, at most 64 tokens
"""

from __future__ import annotations

import ctypes

import torch

from . import OK, SgemmError, lib

Q4_ZEROS = 1
Q4_SCALE_FP16 = 2
MOE_MAX_TOKENS = 64

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _Q4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("group", ctypes.c_int), ("flags", ctypes.c_int)]


class _Moe(ctypes.Structure):
    _fields_ = [("router", ctypes.c_void_p), ("router_dtype", ctypes.c_int),
                ("dtype", ctypes.c_int), ("D", ctypes.c_int), ("F", ctypes.c_int),
                ("E", ctypes.c_int), ("top_k", ctypes.c_int), ("renormalize", ctypes.c_int),
                ("gate", _Q4), ("up", _Q4), ("down", _Q4)]


def _cuda_tensor(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _dtype_code(t, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, not {t.dtype}")
    return code


def _rows(t, name: str, cols: int) -> int:
    """The row pitch of a 2-D tensor whose rows are contiguous and do not overlap."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols:
        raise ValueError(f"{name} must be 2-D with {cols} columns, not {tuple(shape)}")
    rows = shape[0]
    pitch, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and pitch < cols):
        raise ValueError(f"{name} must have contiguous rows that do not overlap "
                         f"(strides {t.stride()})")
    return pitch if rows > 1 else max(pitch, cols)


# The current stream's handle and the current device without the public calls' wrapping,
# which costs a small product's call as much as its launch.
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _result(shape, dtype, device, stream):
    """An empty tensor for a call on ``stream``. It is allocated there: the current stream's
    memory may still be in use by that stream's pending work, which the caller cannot order
    before the call. The caller goes on with the tensor on the current stream, so it is marked
    as in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _launch(fn, what, tensors, index, stream, *args):
    """Calls a library function with a stream as its last argument, on the tensors' device.
    Tensors used on a stream other than the current one are marked as in use there."""
    if stream is None:
        handle = _current_handle(index)
    else:
        handle = stream.cuda_stream
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    if index == _current_device():
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, handle)
    if rc != OK:
        raise SgemmError(rc, what)


class Q4Matrix:
    """A packed 4-bit matrix N x K, or a stack of ``count`` of them; made by q4_quantize or
    q4_pack. ``data`` is the packed buffer (uint8, one dimension)."""

    def __init__(self, N: int, K: int, group: int, zeros: bool, fp16_scales: bool, stack: bool,
                 count: int, device, stream=None):
        self.N, self.K, self.group = int(N), int(K), int(group)
        self.zeros, self.count, self.stack = bool(zeros), int(count), bool(stack)
        self.scale_dtype = torch.float16 if fp16_scales else torch.bfloat16
        flags = (Q4_ZEROS if zeros else 0) | (Q4_SCALE_FP16 if fp16_scales else 0)
        self._c = _Q4(None, self.count, self.N, self.K, self.group, flags)
        self._ref = ctypes.byref(self._c)
        size = lib().sgemm_q4_bytes(self._ref)
        if size < 0:
            raise SgemmError(int(size), f"4-bit matrix {count} x {N} x {K}, group {group}")
        self.data = _result(size, torch.uint8, device, stream)
        self.device = self.data.device
        self.index = self.device.index
        self._c.data = self.data.data_ptr()
        self._matmul = lib().sgemm_q4_matmul

    @property
    def nbytes(self) -> int:
        return self.data.numel()

    @property
    def shape(self):
        return (self.count, self.N, self.K) if self.stack else (self.N, self.K)

    def __repr__(self):
        return (f"Q4Matrix(shape={self.shape}, group={self.group}, zeros={self.zeros}, "
                f"scales={self.scale_dtype}, device={self.device})")


def _packed_for(t, name, group, zeros, fp16_scales, transposed, stream) -> Q4Matrix:
    _cuda_tensor(t, name)
    if t.dim() not in (2, 3) or not t.is_contiguous() or t.numel() == 0:
        raise ValueError(f"{name} must be a contiguous, non-empty 2-D or 3-D tensor")
    N, K = (t.shape[-1], t.shape[-2]) if transposed else (t.shape[-2], t.shape[-1])
    count = t.shape[0] if t.dim() == 3 else 1
    return Q4Matrix(N, K, group, zeros, fp16_scales, t.dim() == 3, count, t.device, stream)


def q4_quantize(B, group: int = 128, zeros: bool = False, transposed: bool = False, stream=None):
    """Rounds B (N x K, or E x N x K) to 4 bits with a bfloat16 scale for every ``group``
    rows of a column, and a zero point with ``zeros``. ``transposed``: B is stored K x N,
    one row for each output. Returns a Q4Matrix."""
    _cuda_tensor(B, "B")
    code = _dtype_code(B, "B")
    W = _packed_for(B, "B", group, zeros, False, transposed, stream)
    _launch(lib().sgemm_q4_quantize, "sgemm_q4_quantize", (B, W.data), W.index, stream,
            B.data_ptr(), code, int(transposed), W._ref)
    return W


def q4_pack(codes, scales, zeros=None, group: int = 128, transposed: bool = False, stream=None):
    """Lays out weights that are quantised already: codes (uint8, 0..15) N x K or
    E x N x K, scales (bfloat16 or float16) and zeros (uint8) with ceil(N / group) in the
    place of N; with ``transposed`` the last two dimensions of all three are exchanged.
    Returns a Q4Matrix."""
    _cuda_tensor(codes, "codes")
    if codes.dtype != torch.uint8:
        raise ValueError("codes must be uint8")
    W = _packed_for(codes, "codes", group, zeros is not None,
                    getattr(scales, "dtype", None) == torch.float16, transposed, stream)
    groups = -(-W.N // W.group)
    shape = codes.shape[:-2] + ((W.K, groups) if transposed else (groups, W.K))
    for name, t, kinds in (("scales", scales, (torch.bfloat16, torch.float16)),
                           ("zeros", zeros, (torch.uint8,))):
        if t is None and name == "zeros":
            continue
        _cuda_tensor(t, name)
        if t.dtype not in kinds or t.shape != shape or not t.is_contiguous() or \
                t.device != codes.device:
            raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} and type "
                             f"{' or '.join(map(str, kinds))} on {codes.device}")
    _launch(lib().sgemm_q4_pack, "sgemm_q4_pack", (codes, scales, zeros, W.data), W.index,
            stream, codes.data_ptr(), scales.data_ptr(),
            None if zeros is None else zeros.data_ptr(), int(transposed), W._ref)
    return W


def q4_dequantize(W: Q4Matrix, out=None, stream=None):
    """The float32 values of W, of shape ``W.shape``."""
    if not isinstance(W, Q4Matrix):
        raise TypeError("W must be a Q4Matrix")
    if out is None:
        out = _result(W.shape, torch.float32, W.device, stream)
    else:
        _cuda_tensor(out, "out")
        if out.dtype != torch.float32 or tuple(out.shape) != W.shape or not out.is_contiguous() \
                or out.device != W.device:
            raise ValueError(f"out must be a contiguous float32 tensor of shape {W.shape} on "
                             f"{W.device}")
    _launch(lib().sgemm_q4_dequantize, "sgemm_q4_dequantize", (W.data, out), W.index, stream,
            W._ref, out.data_ptr())
    return out


def q4_matmul(A, W: Q4Matrix, out=None, stream=None):
    """A (M x N, float32, bfloat16 or float16; a slice of a wider tensor will do) times the
    packed N x K matrix W, for few rows. Returns an M x K tensor of A's type."""
    if not isinstance(W, Q4Matrix):
        raise TypeError("W must be a Q4Matrix")
    if W.stack:
        raise ValueError("W must be a single matrix, not a stack")
    _cuda_tensor(A, "A")
    code = _dtype_code(A, "A")
    lda = _rows(A, "A", W.N)
    M = A.shape[0]
    if A.get_device() != W.index:
        raise ValueError(f"A is on {A.device}, W on {W.device}")
    if out is None:
        out = _result((M, W.K), A.dtype, W.device, stream)
        ldc = W.K
    else:
        _cuda_tensor(out, "out")
        if out.dtype != A.dtype or out.shape[0] != M or out.device != A.device:
            raise ValueError(f"out must be {M} x {W.K} of type {A.dtype} on {A.device}")
        ldc = _rows(out, "out", W.K)
    index = W.index
    if stream is None and index == _current_device():  # the usual call, without a detour
        rc = W._matmul(A.data_ptr(), code, lda, M, W._ref, out.data_ptr(), ldc,
                       _current_handle(index))
        if rc != OK:
            raise SgemmError(rc, "sgemm_q4_matmul")
        return out
    _launch(W._matmul, "sgemm_q4_matmul", (A, W.data, out), index, stream,
            A.data_ptr(), code, lda, M, W._ref, out.data_ptr(), ldc)
    return out


class MoeLayer:
    """A mixture-of-experts layer: router (E x D), gate and up (stacks of E matrices
    D x F) and down (E matrices F x D) as Q4Matrix. Calling it with x (T x D, at most 64
    tokens) gives ``(y, ids, weights)``: y like x, and for each token the ``top_k`` chosen
    experts in ascending order (int32) with their weights (float32). ``live`` (T, bool or
    uint8) marks the tokens to work on; the others get rows of zeros, ids -1, weights 0."""

    def __init__(self, router, gate: Q4Matrix, up: Q4Matrix, down: Q4Matrix, top_k: int,
                 renormalize: bool = True, dtype=None):
        _cuda_tensor(router, "router")
        if router.dim() != 2 or not router.is_contiguous():
            raise ValueError("router must be a contiguous E x D tensor")
        E, D = router.shape
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            if not isinstance(w, Q4Matrix):
                raise TypeError(f"{name} must be a Q4Matrix")
            if w.device != router.device:
                raise ValueError(f"{name} is on {w.device}, router on {router.device}")
        F = gate.K
        for name, w, shape in (("gate", gate, (E, D, F)), ("up", up, (E, D, F)),
                               ("down", down, (E, F, D))):
            if (w.count, w.N, w.K) != shape:
                raise ValueError(f"{name} must be a stack of shape {shape}, not "
                                 f"{(w.count, w.N, w.K)}")
        if gate.group != up.group or gate._c.flags != up._c.flags:
            raise ValueError("gate and up must have the same group size, zero points and scales")
        if not 1 <= top_k <= min(E, 16):
            raise ValueError(f"top_k must lie between 1 and {min(E, 16)}")
        self.router, self.gate, self.up, self.down = router, gate, up, down
        self.top_k, self.renormalize = int(top_k), bool(renormalize)
        self.dtype = router.dtype if dtype is None else dtype
        if self.dtype not in _DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, not {self.dtype}")
        self.E, self.D, self.F, self.device = E, D, F, router.device
        self.index = self.device.index
        self._c = _Moe(router.data_ptr(), _dtype_code(router, "router"), _DTYPES[self.dtype], D, F,
                       E, self.top_k, int(self.renormalize), gate._c, up._c, down._c)
        self._ref = ctypes.byref(self._c)
        self._fn = lib().sgemm_moe

    def __call__(self, x, live=None, out=None, stream=None):
        _cuda_tensor(x, "x")
        if x.dtype is not self.dtype or x.get_device() != self.index:
            raise ValueError(f"x must be {self.dtype} on {self.device}")
        ldx = _rows(x, "x", self.D)
        T = x.shape[0]
        if T > MOE_MAX_TOKENS:
            raise ValueError(f"at most {MOE_MAX_TOKENS} tokens in a call, not {T}")
        if live is not None:
            _cuda_tensor(live, "live")
            if live.dtype not in (torch.bool, torch.uint8) or live.shape != (T,) or \
                    not live.is_contiguous() or live.device != self.device:
                raise ValueError(f"live must be {T} bool or uint8 values on {self.device}")
        if out is None:
            out = _result((T, self.D), self.dtype, self.device, stream)
            ldy = self.D
        else:
            _cuda_tensor(out, "out")
            if out.dtype != x.dtype or out.shape[0] != T or out.device != x.device:
                raise ValueError(f"out must be {T} x {self.D} of type {x.dtype} on {x.device}")
            ldy = _rows(out, "out", self.D)
        ids = _result((T, self.top_k), torch.int32, self.device, stream)
        weights = _result((T, self.top_k), torch.float32, self.device, stream)
        args = (self._ref, x.data_ptr(), ldx, T, None if live is None else live.data_ptr(),
                out.data_ptr(), ldy, ids.data_ptr(), weights.data_ptr())
        index = self.index
        if stream is None and index == _current_device():
            rc = self._fn(*args, _current_handle(index))
            if rc != OK:
                raise SgemmError(rc, "sgemm_moe")
        else:
            _launch(self._fn, "sgemm_moe",
                    (x, live, out, ids, weights, self.router, self.gate.data, self.up.data,
                     self.down.data), index, stream, *args)
        return out, ids, weights
