"""4-bit microscaled matrices, their products, and the gated feed-forward
block in 16 and in 4 bits: argument marshalling for the entry points of
``ddgemm.h`` (formats, layouts and roundings are defined there).

    q = mx4_quantize(x, "mxfp4")            # rows; cols=True: columns
    C = mx4_gemm(a, b)                      # a: M x K, b: N x K, C = a b^T
    y, saved = ff_gated(x, Wg, Wu, Wd, save=True)
    dx, dWg, dWu, dWd = ff_gated_backward(dy, x, Wg, Wu, Wd, saved)
    w_in, w_out = mx4_ff_weights(Wg, Wu, Wd, "mxfp4")
    y = mx4_ff_gated(x, w_in, w_out)
"""
from __future__ import annotations

import ctypes
import dataclasses

import extended_precision_gemm_gb300 as _ddg

MX4_FORMATS = {"mxfp4": 0, "nvfp4": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _torch():
    return _ddg._torch()


def _lookup(table, key, name):
    if key not in table:
        raise ValueError(f"{name} must be one of {', '.join(table)}")
    return table[key]


def _type(dtype, name, sixteen=False):
    torch = _torch()
    types = {torch.bfloat16: 1, torch.float16: 2} if sixteen else {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
    if dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(t) for t in types)}")
    return types[dtype]


def _matrix(t, name, dtype=None):
    """A 2-D CUDA tensor with unit column stride (of `dtype`)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or (dtype is not None and t.dtype != dtype):
        raise TypeError(f"{name} must be a 2-D {dtype or 'torch'} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name} must be on a CUDA device")
    if t.numel() > 0 and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be row-major with unit column stride")
    if t.shape[0] > 1 and t.shape[1] > 0 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t


def _like(out, shape, dtype, device, name, stream):
    """`out` checked, or a new tensor (recorded on `stream`, which may not be
    the one it was allocated for)."""
    torch = _torch()
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        if stream is not None:
            out.record_stream(stream)
        return out
    _matrix(out, name, dtype)
    if tuple(out.shape) != tuple(shape) or out.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} on {device}")
    return out


def _same_device(*tensors):
    if any(t is not None and t.device != tensors[0].device for t in tensors):
        raise ValueError("tensors must be on the same device")


# ---- 4-bit matrices ----

@dataclasses.dataclass
class MX4:
    """A rows x k matrix in 4-bit microscaled form (layout: ddgemm.h).

    codes: uint8 (rows, k / 2 rounded up to 16) or wider, 16-byte rows; scales:
    uint8, the tiles one after the other; exponents: int32 (rows), nvfp4 only.
    """

    codes: object
    scales: object
    exponents: object
    rows: int
    k: int
    fmt: str

    @property
    def shape(self):
        return (self.rows, self.k)

    def _args(self, name):
        torch = _torch()
        fmt = _lookup(MX4_FORMATS, self.fmt, "fmt")
        width, scale_bytes = mx4_layout(self.rows, self.k, self.fmt)
        c, s, e = self.codes, self.scales, self.exponents
        if not isinstance(c, torch.Tensor) or c.dtype != torch.uint8 or c.dim() != 2 or not c.is_cuda:
            raise TypeError(f"{name}.codes must be a 2-D uint8 CUDA tensor")
        if c.shape[0] != self.rows or c.shape[1] < width or (c.numel() > 0 and c.stride(1) != 1):
            raise ValueError(f"{name}.codes must be {self.rows} rows of at least {width} bytes")
        if not isinstance(s, torch.Tensor) or s.dtype != torch.uint8 or not s.is_cuda:
            raise TypeError(f"{name}.scales must be a uint8 CUDA tensor")
        if s.numel() < scale_bytes or not s.is_contiguous():
            raise ValueError(f"{name}.scales must hold {scale_bytes} contiguous bytes")
        if fmt == 1:
            if not isinstance(e, torch.Tensor) or e.dtype != torch.int32 or not e.is_cuda:
                raise TypeError(f"{name}.exponents must be an int32 CUDA tensor")
            if e.numel() < self.rows or not e.is_contiguous():
                raise ValueError(f"{name}.exponents must hold {self.rows} contiguous values")
            _same_device(c, s, e)
        _same_device(c, s)
        ld = c.stride(0) if self.rows > 1 else -(-c.shape[1] // 16) * 16
        return fmt, c.data_ptr(), ld, s.data_ptr(), (e.data_ptr() if fmt == 1 else None)


def mx4_layout(rows: int, k: int, fmt: str = "mxfp4"):
    """(bytes of a row of codes, bytes of all scales) of a rows x k matrix."""
    width, scales = ctypes.c_int64(), ctypes.c_int64()
    _ddg._check("dd_mx4_layout", _ddg.load().dd_mx4_layout(_lookup(MX4_FORMATS, fmt, "fmt"), rows, k,
                                                          ctypes.byref(width), ctypes.byref(scales)))
    return width.value, scales.value


def mx4_quantize(x, fmt: str = "mxfp4", cols: bool = False, out: MX4 | None = None, stream=None) -> MX4:
    """The rows of x (float32, bfloat16 or float16), or with cols its columns,
    in 4-bit form.  A K x N right-hand side is quantised with cols=True."""
    torch = _torch()
    f = _lookup(MX4_FORMATS, fmt, "fmt")
    _matrix(x, "x")
    t = _type(x.dtype, "x")
    rows, k = (x.shape[1], x.shape[0]) if cols else (x.shape[0], x.shape[1])
    if out is None:
        width, scale_bytes = mx4_layout(rows, k, fmt)
        new = lambda *shape, dtype=torch.uint8: torch.empty(shape, dtype=dtype, device=x.device)  # noqa: E731
        out = MX4(new(rows, width), new(scale_bytes), new(rows, dtype=torch.int32) if f else None, rows, k, fmt)
        if stream is not None:
            for part in (out.codes, out.scales) + ((out.exponents,) if f else ()):
                part.record_stream(stream)
    elif out.shape != (rows, k) or out.fmt != fmt:
        raise ValueError(f"out must be a {rows} x {k} {fmt} matrix")
    _, codes, ldq, scales, exponents = out._args("out")
    _same_device(x, out.codes)
    _ddg._check("dd_mx4_quantize", _ddg.load().dd_mx4_quantize(
        f, t, int(cols), rows, k, x.data_ptr(), _ddg._ld(x), codes, ldq, scales, exponents, _ddg._stream_handle(stream)))
    return out


def mx4_dequantize(q: MX4, dtype=None, out=None, stream=None):
    """The values q stands for, as a rows x k tensor (bfloat16 by default, which holds them exactly)."""
    torch = _torch()
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    t = _type(dtype, "dtype")
    f, codes, ldq, scales, exponents = q._args("q")
    out = _like(out, q.shape, dtype, q.codes.device, "out", stream)
    _ddg._check("dd_mx4_dequantize", _ddg.load().dd_mx4_dequantize(
        f, t, q.rows, q.k, codes, ldq, scales, exponents, out.data_ptr(), _ddg._ld(out), _ddg._stream_handle(stream)))
    return out


def mx4_tile_scales(scales, fmt: str = "mxfp4"):
    """Scale bytes (rows, blocks) in the tiled order of ddgemm.h, padded with
    zeros: for matrices quantised elsewhere, once when they are loaded."""
    torch = _torch()
    per_k = 2 * (4 if _lookup(MX4_FORMATS, fmt, "fmt") == 0 else 8)  # blocks in 256 of k
    rows, blocks = scales.shape
    s = torch.nn.functional.pad(scales, (0, -blocks % per_k, 0, -rows % 128))
    return s.view(s.shape[0] // 128, 4, 32, -1, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def mx4_gemm(a: MX4, b: MX4, dtype=None, out=None, alpha: float = 1.0, stream=None):
    """alpha a b^T for 4-bit matrices a (M x K) and b (N x K) of one format, as
    an M x N tensor (bfloat16 by default)."""
    torch = _torch()
    if a.fmt != b.fmt or a.k != b.k:
        raise ValueError("a and b must share format and k")
    dtype = dtype or (out.dtype if out is not None else torch.bfloat16)
    t = _type(dtype, "dtype")
    f, ac, lda, as_, ae = a._args("a")
    _, bc, ldb, bs, be = b._args("b")
    _same_device(a.codes, b.codes)
    out = _like(out, (a.rows, b.rows), dtype, a.codes.device, "out", stream)
    _ddg._check("dd_mx4_gemm", _ddg.load().dd_mx4_gemm(
        f, a.rows, b.rows, a.k, ac, lda, as_, ae, bc, ldb, bs, be, alpha, t, out.data_ptr(), _ddg._ld(out),
        _ddg._stream_handle(stream)))
    return out


# ---- the gated block ----

def _ff_shapes(x, Wg, Wu, Wd):
    for t, n in ((x, "x"), (Wg, "Wg"), (Wu, "Wu"), (Wd, "Wd")):
        _matrix(t, n, x.dtype if n != "x" else None)
    code = _type(x.dtype, "x", sixteen=True)
    T, D = x.shape
    F = Wg.shape[0]
    if tuple(Wg.shape) != (F, D) or tuple(Wu.shape) != (F, D) or tuple(Wd.shape) != (D, F):
        raise ValueError("Wg and Wu must be F x D and Wd D x F for x of T x D")
    _same_device(x, Wg, Wu, Wd)
    return code, T, D, F


def ff_gated_saved_size(T: int, F: int, dtype) -> int:
    """Bytes that ff_gated(save=True) keeps for the backward pass."""
    n = ctypes.c_size_t()
    _ddg._check("dd_ff_gated_saved_size", _ddg.load().dd_ff_gated_saved_size(_type(dtype, "dtype", sixteen=True), T, F,
                                                                            ctypes.byref(n)))
    return n.value


def ff_gated(x, Wg, Wu, Wd, act: str = "silu", save: bool = False, out=None, stream=None):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T in bfloat16 or float16 (x: T x D, Wg and
    Wu: F x D, Wd: D x F); with save=True (y, saved) for ff_gated_backward."""
    torch = _torch()
    code, T, D, F = _ff_shapes(x, Wg, Wu, Wd)
    a = _lookup(ACTIVATIONS, act, "act")
    y = _like(out, (T, D), x.dtype, x.device, "out", stream)
    saved, n = None, 0
    if save:
        n = ff_gated_saved_size(T, F, x.dtype)
        saved = torch.empty(n, dtype=torch.uint8, device=x.device)
        if stream is not None:
            saved.record_stream(stream)
    ld = _ddg._ld
    _ddg._check("dd_ff_gated", _ddg.load().dd_ff_gated(
        code, a, T, D, F, x.data_ptr(), ld(x), Wg.data_ptr(), ld(Wg), Wu.data_ptr(), ld(Wu), Wd.data_ptr(), ld(Wd),
        y.data_ptr(), ld(y), saved.data_ptr() if n else None, n, _ddg._stream_handle(stream)))
    return (y, saved) if save else y


def ff_gated_backward(dy, x, Wg, Wu, Wd, saved, dx=None, dWg=None, dWu=None, dWd=None, need=(True,) * 4, stream=None):
    """(dx, dWg, dWu, dWd) from dy and what ff_gated(save=True) kept; `need` says
    which of them are wanted (None in the place of the others).  Tensors that
    are given are overwritten."""
    torch = _torch()
    code, T, D, F = _ff_shapes(x, Wg, Wu, Wd)
    _matrix(dy, "dy", x.dtype)
    if tuple(dy.shape) != (T, D):
        raise ValueError("dy must be T x D")
    if not isinstance(saved, torch.Tensor) or saved.dtype != torch.uint8 or not saved.is_cuda or not saved.is_contiguous():
        raise TypeError("saved must be the uint8 CUDA tensor that ff_gated returned")
    if saved.numel() != ff_gated_saved_size(T, F, x.dtype):
        raise ValueError("saved is of another T, F or type")
    _same_device(x, dy, saved)
    shapes = (("dx", dx, (T, D)), ("dWg", dWg, (F, D)), ("dWu", dWu, (F, D)), ("dWd", dWd, (D, F)))
    outs = [_like(o, shape, x.dtype, x.device, n, stream) if want else None for (n, o, shape), want in zip(shapes, need)]
    ld = _ddg._ld
    args = []
    for o, (_, _, shape) in zip(outs, shapes):
        args += [o.data_ptr(), ld(o)] if o is not None else [None, max(shape[1], 1)]
    _ddg._check("dd_ff_gated_backward", _ddg.load().dd_ff_gated_backward(
        code, T, D, F, dy.data_ptr(), ld(dy), x.data_ptr(), ld(x), Wg.data_ptr(), ld(Wg), Wu.data_ptr(), ld(Wu),
        Wd.data_ptr(), ld(Wd), saved.data_ptr() if saved.numel() else None, saved.numel(), *args,
        _ddg._stream_handle(stream)))
    return tuple(outs)


def mx4_ff_weights(Wg, Wu, Wd, fmt: str = "mxfp4", stream=None):
    """(w_in, w_out), the weights of mx4_ff_gated from those of ff_gated, once
    when a model is loaded: Wg and Wu in one matrix, 32 rows of each in turn
    (the last groups filled up with zeros), quantised along D, and Wd
    quantised along F."""
    torch = _torch()
    F, D = Wg.shape
    if tuple(Wu.shape) != (F, D) or tuple(Wd.shape) != (D, F):
        raise ValueError("Wg and Wu must be F x D and Wd D x F")
    pair = [torch.nn.functional.pad(w, (0, 0, 0, -F % 32)).view(-1, 32, D) for w in (Wg, Wu)]
    both = torch.stack(pair, 1).view(-1, D)
    return mx4_quantize(both, fmt, stream=stream), mx4_quantize(_matrix(Wd, "Wd"), fmt, stream=stream)


def mx4_ff_gated(x, w_in: MX4, w_out: MX4, act: str = "silu", out=None, stream=None):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T with 4-bit operands: the weights as
    mx4_ff_weights lays them out, x and the hidden values quantised in the
    call.  x and y: float32, bfloat16 or float16, T x D."""
    _matrix(x, "x")
    t = _type(x.dtype, "x")
    a = _lookup(ACTIVATIONS, act, "act")
    T, D = x.shape
    F = w_out.k
    if w_in.fmt != w_out.fmt or w_in.k != D or w_out.rows != D or w_in.rows != 2 * (-(-F // 32) * 32):
        raise ValueError("w_in must be 2 * (F rounded up to 32) x D and w_out D x F, of one format")
    f, ic, ldi, is_, ie = w_in._args("w_in")
    _, oc, ldo, os_, oe = w_out._args("w_out")
    _same_device(x, w_in.codes, w_out.codes)
    y = _like(out, (T, D), x.dtype, x.device, "out", stream)
    _ddg._check("dd_mx4_ff_gated", _ddg.load().dd_mx4_ff_gated(
        f, t, a, T, D, F, x.data_ptr(), _ddg._ld(x), ic, ldi, is_, ie, oc, ldo, os_, oe, y.data_ptr(), _ddg._ld(y),
        _ddg._stream_handle(stream)))
    return y
