"""The norm in front of a layer's products, rows in 4-bit blocks and their products, through the
C ABI of include/sparse_ffn_mx4.h. torch supplies device memory and streams; every step runs in
the library.

    wq, ws = quantize_mx4(w)                       # a weight matrix [N, K], offline
    q, s, r = rms_norm(x, g, residual=r, out="mx4")
    y = mx4_matmul(q, wq, ws, x_scale=s)           # y = norm(x + r) W^T

    q, s, r = rms_norm(x, g, residual=r, out="i8")
    y = i8_matmul(q, w8, w8_scale, x_scale=s)      # the same with 8-bit rows

There are no gradients. Rows in 4-bit blocks are two uint8 tensors: codes [..., 16 B] and scales
[..., B] for B blocks of 32 numbers; quantize_mx4 lays them out as the products read them. Tensors
given for outputs must not overlap the inputs unless it is said. A call with `stream` goes to that
stream and takes its outputs from that stream's memory: use them elsewhere only in order after it,
and keep the inputs until it is done, or record_stream them.

Calls on the current device and stream whose tensors lie as the library reads them go through the
extension module _calls (csrc/sffn_calls.cpp), which does in one step what the functions here do: a
third to a half of the host's time. Where it returns None the function goes on here, with copies,
another stream or device, given outputs, or the error; so does every call where there is no such module
that was built for this Python and torch.
"""
from __future__ import annotations

import warnings
from typing import Optional, Tuple, Union

import torch

from . import _native as N
from .experts import _F32, _I8, _TYPES, _U8, _on, _out, _out_dtype, _type, _vector, _work
from .experts import _current, _rows as _some_rows


class _Without:
    """In the place of _calls: leaves every call to the functions here."""

    norm = quantize = dequantize = matmul = staticmethod(lambda *a: None)


def _short_way():
    try:
        from . import _calls
    except ImportError as e:
        why = str(e)
    else:
        built_for = getattr(_calls, "built_for", None)
        if built_for == str(torch.__version__):
            _calls.bind(*(N.address(f) for f in ("sparse_ffn_rms_norm", "sparse_ffn_quantize_mx4",
                                                 "sparse_ffn_dequantize_mx4", "sparse_ffn_mx4_matmul_work_bytes",
                                                 "sparse_ffn_mx4_matmul")))
            return _calls
        why = f"built for torch {built_for}, not {torch.__version__}"
    warnings.warn(f"the extension module _calls is not used ({why}): calls of mx4.py take longer on the host. "
                  "activation_sparse_decode_rank_amd/build.py builds it", RuntimeWarning)
    return _Without


_calls = _short_way()
# the current device's number, without the checks around it where torch offers that
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_OUT = {None: -1, **_TYPES, "i8": N.SFFN_I8, "mx4": N.SFFN_MX4}


def _done(got, what: str):
    """What _calls returned: outputs, or a status."""
    if type(got) is int:
        raise N.SparseFFNError(got, what)
    return got


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """Rows and row distance of a matrix whose rows are contiguous; of no rows, whatever the strides."""
    return (0, t.shape[1]) if t.dim() == 2 and t.shape[0] == 0 else _some_rows(t, name)


def _flat(x: torch.Tensor, stream) -> torch.Tensor:
    """x [..., K] as a matrix whose rows are contiguous; a copy, made where the call runs, only
    where there is no such view."""
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must have rows of at least one value")
    if x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] == 1) and (x.shape[0] <= 1 or x.stride(0) >= x.shape[1]):
        return x
    if x.is_contiguous():
        return x.view(-1, x.shape[-1])
    with torch.cuda.stream(stream):
        return x.contiguous().view(-1, x.shape[-1])


def _blocks(q: torch.Tensor, scale: torch.Tensor, dev, name: str) -> Tuple[int, int, int, int]:
    """Rows, blocks and row distances (codes, scales) of two-dimensional rows in 4-bit blocks."""
    if q.dtype != _U8 or scale.dtype != _U8 or q.device != dev or scale.device != dev:
        raise ValueError(f"{name} and its scales must be uint8 on {dev}")
    if q.dim() != 2 or scale.dim() != 2:
        raise ValueError(f"{name} and its scales must have two dimensions")
    R, n = q.shape
    if scale.shape[0] != R or n != 16 * scale.shape[1] or n == 0:
        raise ValueError(f"{name} [{R}, {n}] must be codes [R, 16 B] with scales [R, B]")
    B = n // 16
    room = (B + 15) // 16 * 16
    ldq, oq = q.stride()
    lds, os_ = scale.stride()
    if R and (oq != 1 or (os_ != 1 and B > 1)):
        raise ValueError(f"the rows of {name} and of its scales must be contiguous")
    if R <= 1:
        ldq, lds = n, room
    if ldq % 16 or ldq < n or q.data_ptr() % 16:
        raise ValueError(f"the rows of {name} must begin at multiples of 16 bytes")
    if lds % 16 or lds < B or scale.data_ptr() % 16:
        raise ValueError(f"the rows of {name}'s scales must begin at multiples of 16 bytes "
                         "(quantize_mx4 lays them out so)")
    if B != room and R and scale.storage_offset() + (R - 1) * lds + room > scale.untyped_storage().nbytes():
        raise ValueError(f"{name}'s scales end inside 16 bytes: their rows need room up to the next "
                         "multiple of 16 (quantize_mx4 lays them out so)")
    return R, B, ldq, lds


def _new_blocks(on, shape, K: int):
    """Room for rows [*shape, K] in 4-bit blocks: codes, scales, and the scales' row distance."""
    B = (K + 31) // 32
    lds = (B + 15) // 16 * 16
    q = on.empty((*shape, 16 * B), _U8)
    scale = on.empty((*shape, lds), _U8)
    return q, (scale if lds == B else scale[..., :B]), lds


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, *,
             residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             out: Union[None, str, torch.dtype] = None, residual_out: Optional[torch.Tensor] = None,
             stream=None):
    """The root-mean-square norm of the rows of x ([..., d]), v w / sqrt(mean(v^2) + eps), with v = x
    or, where a residual is given, x + residual rounded to x's type (sparse_ffn_rms_norm).

    weight: [d], any float type (None: 1). out: a float type (default x's): returns y; "i8": returns
    8-bit rows and their scales, as quantize_rows gives them for the float32 y and i8_matmul takes
    them; "mx4": returns codes and scales, as quantize_mx4 gives them for the float32 y and
    mx4_matmul takes them. With a residual (x's shape and type) v comes last, in residual_out where
    that is given: it may be the residual itself, or x."""
    kind = _OUT.get(out)
    i = x.device.index
    if kind is not None and stream is None and i is not None and i == _device():
        got = _calls.norm(x, weight, residual, eps, kind, residual_out, i, _current(i))
        if got is not None:
            return _done(got, "sparse_ffn_rms_norm")
    dt = _type(x, "x")
    if out is None:
        out, kind = x.dtype, dt
    if kind is None:
        raise ValueError("out must be float32, float16, bfloat16, 'i8' or 'mx4'")
    if (residual is None) and residual_out is not None:
        raise ValueError("residual_out belongs to a residual")
    with _on(x, stream) as on:
        dev = on.device
        flat = _flat(x, stream)
        shape, d = x.shape[:-1], x.shape[-1]
        R, ldx = _rows(flat, "x")
        wp, wt = None, 0
        if weight is not None:
            wt = _type(weight, "weight")
            wp = _vector(weight, (d,), weight.dtype, dev, "weight")
        rp = sp = None
        ldr = lds_ = d
        if residual is not None:
            if residual.shape != x.shape or residual.dtype != x.dtype or residual.device != dev:
                raise ValueError(f"residual must be {x.dtype} of shape {tuple(x.shape)} on {dev}")
            rflat = _flat(residual, stream)
            ldr = _rows(rflat, "residual")[1]
            rp = rflat.data_ptr()
            if residual_out is None:
                residual_out = on.empty(x.shape, x.dtype)
                sp = residual_out.data_ptr()
            else:
                _out(residual_out, on, x.shape, x.dtype, "residual_out")
                if residual_out.dim() != 2 and not residual_out.is_contiguous():
                    raise ValueError("residual_out must be contiguous, or a matrix of contiguous rows")
                lds_ = _rows(residual_out if residual_out.dim() == 2 else residual_out.view(-1, d),
                             "residual_out")[1]
                sp = residual_out.data_ptr()
        scale, lds, sc = None, 0, None
        if kind == N.SFFN_I8:
            ldy = (d + 15) // 16 * 16
            y = on.empty((*shape, ldy), _I8)
            scale = on.empty(shape, _F32)
        elif kind == N.SFFN_MX4:
            y, scale, lds = _new_blocks(on, shape, d)
            ldy = y.shape[-1]
        else:
            ldy = d
            y = on.empty(x.shape, out)
        if scale is not None:
            sc = scale.data_ptr()
        N.sparse_ffn_rms_norm(flat.data_ptr(), dt, ldx, rp, ldr, R, d, wp, wt, eps, sp, lds_,
                              y.data_ptr(), kind, ldy, sc, lds, on.handle)
    if kind == N.SFFN_I8 and ldy != d:
        y = y[..., :d]
    if residual is None:
        return y if scale is None else (y, scale)
    return (y, residual_out) if scale is None else (y, scale, residual_out)


def quantize_mx4(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of x ([..., K]) in 4-bit blocks of 32: codes (uint8 [..., 16 B], two a byte) and
    scales (uint8 [..., B]), B = ceil(K / 32) (sparse_ffn_quantize_mx4). The scales' rows begin at
    multiples of 16 bytes, as the products want them."""
    i = x.device.index
    if stream is None and i is not None and i == _device():
        got = _calls.quantize(x, i, _current(i))
        if got is not None:
            return _done(got, "sparse_ffn_quantize_mx4")
    dt = _type(x, "x")
    with _on(x, stream) as on:
        flat = _flat(x, stream)
        K = x.shape[-1]
        R, ldx = _rows(flat, "x")
        q, scale, lds = _new_blocks(on, x.shape[:-1], K)
        N.sparse_ffn_quantize_mx4(flat.data_ptr(), dt, ldx, R, K, q.data_ptr(), q.shape[-1],
                                  scale.data_ptr(), lds, on.handle)
    return q, scale


def dequantize_mx4(q: torch.Tensor, scale: torch.Tensor, *, cols: Optional[int] = None,
                   dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values that rows in 4-bit blocks stand for (sparse_ffn_dequantize_mx4): [..., cols] of
    dtype, cols at most 32 for each block (the default)."""
    dt = _TYPES.get(dtype)
    i = q.device.index
    if dt is not None and stream is None and i is not None and i == _device():
        got = _calls.dequantize(q, scale, cols, dt, i, _current(i))
        if got is not None:
            return _done(got, "sparse_ffn_dequantize_mx4")
    if dt is None:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    if q.dim() < 1 or scale.dim() != q.dim() or q.shape[:-1] != scale.shape[:-1]:
        raise ValueError("q must be codes [..., 16 B] with scales [..., B]")
    with _on(q, stream) as on:
        shape = q.shape[:-1]
        q2, s2 = q, scale
        if q.dim() != 2:
            q2 = _merged(q, "q") if q.dim() > 2 else q.unsqueeze(0)
            s2 = _merged(scale, "q's scales") if q.dim() > 2 else scale.unsqueeze(0)
        R, B, ldq, lds = _blocks(q2, s2, on.device, "q")
        if cols is None:
            cols = 32 * B
        elif not 32 * (B - 1) < cols <= 32 * B:
            raise ValueError(f"{B} blocks hold rows of {32 * (B - 1) + 1} to {32 * B} values, not {cols}")
        y = on.empty((*shape, cols), dtype)
        N.sparse_ffn_dequantize_mx4(q2.data_ptr(), ldq, s2.data_ptr(), lds, R, cols, y.data_ptr(), dt,
                                    cols, on.handle)
    return y


def _merged(t: torch.Tensor, name: str) -> torch.Tensor:
    """t [..., n] as a matrix of rows that all lie the same distance apart, without a copy."""
    if 0 in t.shape:
        return t.new_empty((0, t.shape[-1]))
    ld, rows = None, 1
    for i in range(t.dim() - 2, -1, -1):
        n = t.shape[i]
        if n == 1:
            continue
        if ld is None:
            ld = t.stride(i)
        elif t.stride(i) != ld * rows:
            raise ValueError(f"the rows of {name} must lie the same distance apart")
        rows *= n
    return t.as_strided((rows, t.shape[-1]), (t.shape[-1] if ld is None else ld, t.stride(-1)))


def mx4_matmul(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, *,
               x_scale: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, y=None, work=None,
               stream=None) -> torch.Tensor:
    """y = x W^T + bias with W in 4-bit blocks (codes w [N, 16 B], w_scale [N, B], as quantize_mx4
    makes them) (sparse_ffn_mx4_matmul). x: float rows [M, K] with ceil(K / 32) = B, which the call
    holds in 4-bit blocks first, or codes [M, 16 B] with x_scale [M, B]. out_dtype: float32,
    float16 or bfloat16 (default: x's type; float32 for codes). work: uint8 scratch (allocated here
    when None); calls that share one must be ordered."""
    kind = _OUT.get(out_dtype)
    i = x.device.index
    if kind is not None and stream is None and y is None and work is None and i is not None and i == _device():
        got = _calls.matmul(x, w, w_scale, x_scale, bias, kind, i, _current(i))
        if got is not None:
            return _done(got, "sparse_ffn_mx4_matmul")
    mx4 = x.dtype == _U8
    if mx4 != (x_scale is not None):
        raise ValueError("x_scale belongs to rows in 4-bit blocks, and they need it")
    dt = N.SFFN_MX4 if mx4 else _type(x, "x")
    out_dtype, yt = _out_dtype(out_dtype, y, _F32 if mx4 else x.dtype)
    with _on(x, stream) as on:
        dev = on.device
        n, B, ldw, ldws = _blocks(w, w_scale, dev, "w")
        if mx4:
            M, bx, ldx, ldxs = _blocks(x, x_scale, dev, "x")
            K, xs = 32 * B, x_scale.data_ptr()
            if bx != B:
                raise ValueError(f"x has {bx} blocks a row, w {B}")
        else:
            M, ldx = _rows(x, "x")
            K, xs, ldxs = x.shape[1], None, 0
            if (K + 31) // 32 != B:
                raise ValueError(f"w's {B} blocks a row do not hold x's {K} values")
        b = None if bias is None else _vector(bias, (n,), _F32, dev, "bias")
        if y is None:
            y, ldy = on.empty((M, n), out_dtype), n
        else:
            y = _out(y, on, (M, n), out_dtype, "y")
            ldy = _rows(y, "y")[1]
        if work is None:
            need = N.sparse_ffn_mx4_matmul_work_bytes(dt, M, n, K)
            if need > 1 << 62:
                raise N.SparseFFNError(N.SFFN_ERR_UNSUPPORTED, "sparse_ffn_mx4_matmul")
            if need:
                work = on.empty(need, _U8)
        else:
            work = _work(work, on)
        N.sparse_ffn_mx4_matmul(x.data_ptr(), dt, xs, ldx, ldxs, M, K, w.data_ptr(), ldw,
                                w_scale.data_ptr(), ldws, b, n, y.data_ptr(), yt, ldy,
                                None if work is None else work.data_ptr(),
                                0 if work is None else work.numel(), on.handle)
    return y
