"""The 8-bit linear layer: activations kept as int8 row codes from the forward
pass to the backward pass, the products that read those codes, and the gated
activation between two layers.

The ``qc_`` functions carry the C ABI's names and arguments (``include/qcodec.h``
states the arithmetic).  The functions without the prefix take tensors only: they
read the sizes from the shapes, allocate the results and the workspace on the
stream they run on, and return the results.

    x_codes, x_scale = rowwise_int8(x)                    # [T, K], kept for the backward pass
    y = int8_matmul(x_codes, x_scale, w_codes, w_scale)   # [T, N]
    dx = int8_input_grad(dy, w_codes, w_scale)            # [T, K]
    dw, _ = int8_weight_grad(dy, x_codes, x_scale)        # [N, K], flat for encode_ef

The backward pass is called as it stands here: as elsewhere in this package no call records
anything for autograd, and results never require a gradient.
"""
from __future__ import annotations

import contextlib
import warnings

import torch

from . import build
from . import (QC_ACCUMULATE_INTO_OUT, QC_DTYPE_BF16, QC_DTYPE_F32, _check, _need, _on_device, _ptr,
               _stream, lib)



class _Declines:
    """In the binding's place where there is none: every call declines, and the code here makes
    the same C call through ctypes."""

    def __getattr__(self, name):
        return lambda *args: None


def _binding():
    why = "it was compiled against another torch or Python"
    if build.bind_fits():
        try:
            from . import _qcbind
            return _qcbind
        except ImportError as e:
            why = str(e)
    warnings.warn(f"the 8-bit layer's calls go through ctypes, at about 10 us more each: the binding {build.BIND_PATH} "
                  f"does not load ({why}); build it with `python {build.__file__}`", RuntimeWarning, stacklevel=2)
    return _Declines()


_qcbind = _binding()

_I8 = (torch.int8,)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16,)
_CODE_OF = {torch.float32: QC_DTYPE_F32, torch.bfloat16: QC_DTYPE_BF16}
_TYPE_OF = {QC_DTYPE_F32: _F32, QC_DTYPE_BF16: _BF16}


def _span(rows, dim, stride, esize):
    return ((rows - 1) * stride + dim) * esize if rows else 0


def _matrix(t, name, rows, dim, stride, dtype):
    """A strided matrix argument of the C ABI: type, dense rows, span."""
    if dtype not in _TYPE_OF:
        return  # the library refuses it
    _need(t, name, _span(rows, dim, stride, 4 if dtype == QC_DTYPE_F32 else 2), _TYPE_OF[dtype], flat=False)
    if rows > 1 and t is not None and not isinstance(t, int) and t.dim() == 2 and t.stride(0) != stride:
        raise ValueError(f"{name}'s row stride ({t.stride(0)}) differs from the stride passed ({stride})")


def _device_of(**tensors):
    """The last check of a call, and the device it runs on: every tensor argument lives on one
    and the same CUDA device, which is current inside the context that this returns.
    (Addresses say nothing about their device: a call with nothing but those runs on
    the current one.)"""
    _on_device(**tensors)
    first, index = None, None
    for name, t in tensors.items():
        if t is None or isinstance(t, int):
            continue
        if index is None:
            first, index = name, t.get_device()
        elif t.get_device() != index:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, {first} on cuda:{index}")
    if index is None or index == torch._C._cuda_getDevice():
        return contextlib.nullcontext()
    return torch.cuda.device(index)


# ----------------------------------------------------------------- the C ABI

def qc_rowwise_int8(x, dtype, x_stride, rows, dim, codes, row_scale, stream=None):
    """Rows of fp32 or bf16 -> int8 codes and one power-of-two scale per row."""
    device = contextlib.nullcontext()
    if rows:
        _matrix(x, "x", rows, dim, x_stride, dtype)
        _need(codes, "codes", rows * dim, _I8)
        _need(row_scale, "row_scale", 4 * rows, _F32)
        device = _device_of(x=x, codes=codes, row_scale=row_scale)
    with device:
        _check(lib.qc_rowwise_int8(_ptr(x), dtype, x_stride, rows, dim, _ptr(codes), _ptr(row_scale),
                                   _stream(stream)))


def qc_rowwise_int8_dequant(codes, row_scale, rows, dim, out, out_dtype, out_stride, stream=None):
    """Row codes -> fp32 or bf16 rows."""
    device = contextlib.nullcontext()
    if rows:
        _need(codes, "codes", rows * dim, _I8)
        _need(row_scale, "row_scale", 4 * rows, _F32)
        _matrix(out, "out", rows, dim, out_stride, out_dtype)
        device = _device_of(codes=codes, row_scale=row_scale, out=out)
    with device:
        _check(lib.qc_rowwise_int8_dequant(_ptr(codes), _ptr(row_scale), rows, dim, _ptr(out), out_dtype,
                                           out_stride, _stream(stream)))


def qc_int8_matmul_workspace(T, N, K) -> int:
    """Bytes of workspace that qc_int8_matmul needs."""
    return int(lib.qc_int8_matmul_workspace(T, N, K))


def qc_int8_matmul_codes_workspace(x_codes, w_codes, T, N, K) -> int:
    """The same for codes where these lie (tensors or addresses)."""
    return int(lib.qc_int8_matmul_codes_workspace(_ptr(x_codes), _ptr(w_codes), T, N, K))


def qc_int8_input_grad_workspace(T, N, K) -> int:
    """Bytes of workspace that qc_int8_input_grad needs."""
    return int(lib.qc_int8_input_grad_workspace(T, N, K))


def qc_int8_weight_grad_workspace(T, N, K) -> int:
    """Bytes of workspace that qc_int8_weight_grad needs."""
    return int(lib.qc_int8_weight_grad_workspace(T, N, K))


def qc_int8_matmul(x_codes, x_scale, w_codes, w_scale, bias, T, N, K, y, y_dtype, y_stride, workspace,
                   workspace_bytes, stream=None):
    """y = (x_codes w_codes^T) with a scale per token and per output channel, plus bias."""
    device = contextlib.nullcontext()
    if T:
        _need(x_codes, "x_codes", T * K, _I8)
        _need(x_scale, "x_scale", 4 * T, _F32)
        _need(w_codes, "w_codes", N * K, _I8)
        _need(w_scale, "w_scale", 4 * N, _F32)
        _need(bias, "bias", 4 * N, _F32)
        _matrix(y, "y", T, N, y_stride, y_dtype)
        _need(workspace, "workspace", workspace_bytes)
        device = _device_of(x_codes=x_codes, x_scale=x_scale, w_codes=w_codes, w_scale=w_scale, bias=bias, y=y,
                            workspace=workspace)
    with device:
        _check(lib.qc_int8_matmul(_ptr(x_codes), _ptr(x_scale), _ptr(w_codes), _ptr(w_scale), _ptr(bias), T, N,
                                  K, _ptr(y), y_dtype, y_stride, _ptr(workspace), workspace_bytes,
                                  _stream(stream)))


def qc_int8_input_grad(dy, dy_stride, w_codes, w_scale, T, N, K, dx, dx_dtype, dx_stride, workspace,
                       workspace_bytes, stream=None):
    """dx = dy (w_codes * w_scale)."""
    device = contextlib.nullcontext()
    if T:
        _matrix(dy, "dy", T, N, dy_stride, QC_DTYPE_BF16)
        _need(w_codes, "w_codes", N * K, _I8)
        _need(w_scale, "w_scale", 4 * N, _F32)
        _matrix(dx, "dx", T, K, dx_stride, dx_dtype)
        _need(workspace, "workspace", workspace_bytes)
        device = _device_of(dy=dy, w_codes=w_codes, w_scale=w_scale, dx=dx, workspace=workspace)
    with device:
        _check(lib.qc_int8_input_grad(_ptr(dy), dy_stride, _ptr(w_codes), _ptr(w_scale), T, N, K, _ptr(dx),
                                      dx_dtype, dx_stride, _ptr(workspace), workspace_bytes, _stream(stream)))


def qc_int8_weight_grad(dy, dy_stride, x_codes, x_scale, T, N, K, dw, dw_dtype, dbias, flags, workspace,
                        workspace_bytes, stream=None):
    """dw = dy^T (x_codes * x_scale), dbias = column sums of dy (dbias may be None)."""
    if T:
        _matrix(dy, "dy", T, N, dy_stride, QC_DTYPE_BF16)
        _need(x_codes, "x_codes", T * K, _I8)
        _need(x_scale, "x_scale", 4 * T, _F32)
    if dw_dtype in _TYPE_OF:
        _need(dw, "dw", N * K * (4 if dw_dtype == QC_DTYPE_F32 else 2), _TYPE_OF[dw_dtype])
    _need(dbias, "dbias", 4 * N, _F32)
    _need(workspace, "workspace", workspace_bytes)
    device = _device_of(dy=dy, x_codes=x_codes, x_scale=x_scale, dw=dw, dbias=dbias, workspace=workspace)
    with device:
        _check(lib.qc_int8_weight_grad(_ptr(dy), dy_stride, _ptr(x_codes), _ptr(x_scale), T, N, K, _ptr(dw),
                                       dw_dtype, _ptr(dbias), flags, _ptr(workspace), workspace_bytes,
                                       _stream(stream)))


def qc_swiglu_encode(gate_up, dtype, stride, rows, dim, h_codes, h_scale, saved_codes, saved_scale,
                     stream=None):
    """h = silu(gate) * up as row codes, and the row codes of gate and up."""
    device = contextlib.nullcontext()
    if rows:
        _matrix(gate_up, "gate_up", rows, 2 * dim, stride, dtype)
        _need(h_codes, "h_codes", rows * dim, _I8)
        _need(h_scale, "h_scale", 4 * rows, _F32)
        _need(saved_codes, "saved_codes", 2 * rows * dim, _I8)
        _need(saved_scale, "saved_scale", 8 * rows, _F32)
        device = _device_of(gate_up=gate_up, h_codes=h_codes, h_scale=h_scale, saved_codes=saved_codes,
                            saved_scale=saved_scale)
    with device:
        _check(lib.qc_swiglu_encode(_ptr(gate_up), dtype, stride, rows, dim, _ptr(h_codes), _ptr(h_scale),
                                    _ptr(saved_codes), _ptr(saved_scale), _stream(stream)))


def qc_swiglu_backward(dh, dtype, dh_stride, saved_codes, saved_scale, rows, dim, dgate_up,
                       dgate_up_stride, stream=None):
    """The gradients by gate and up, from their row codes."""
    device = contextlib.nullcontext()
    if rows:
        _matrix(dh, "dh", rows, dim, dh_stride, dtype)
        _need(saved_codes, "saved_codes", 2 * rows * dim, _I8)
        _need(saved_scale, "saved_scale", 8 * rows, _F32)
        _matrix(dgate_up, "dgate_up", rows, 2 * dim, dgate_up_stride, dtype)
        device = _device_of(dh=dh, saved_codes=saved_codes, saved_scale=saved_scale, dgate_up=dgate_up)
    with device:
        _check(lib.qc_swiglu_backward(_ptr(dh), dtype, dh_stride, _ptr(saved_codes), _ptr(saved_scale), rows,
                                      dim, _ptr(dgate_up), dgate_up_stride, _stream(stream)))


# -------------------------------------------------------------- conveniences
#
# Plainly right arguments (dense tensors of the expected types and shapes on a CUDA
# device) go through the compiled binding, which allocates and calls the library
# without Python in between.  Where it declines (None), the code here looks closer:
# it accepts a strided matrix and says what is wrong with anything else.  Without a
# binding it makes every call.


def _rows(t, name, dtypes):
    """A matrix whose rows are dense: its row stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected one of {tuple(dtypes)}")
    r, d = t.shape
    if d > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be dense along its last dimension")
    stride = t.stride(0) if r > 1 else d
    if stride < d:
        raise ValueError(f"{name}'s rows overlap (row stride {stride}, row length {d})")
    return stride


def _dense(t, name, dtypes, shape):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be a tensor of shape {shape} and dtype {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _codes(codes, scale, what):
    """Row codes and their scales."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
        raise ValueError(f"{what}_codes must be a 2-D tensor")
    shape = tuple(codes.shape)
    _dense(codes, f"{what}_codes", _I8, shape)
    _dense(scale, f"{what}_scale", _F32, (shape[0],))


def _dtype(dtype):
    if dtype not in _CODE_OF:
        raise ValueError(f"dtype {dtype} is not torch.float32 or torch.bfloat16")
    return _CODE_OF[dtype]


def _on(stream, t):
    """Results and workspaces belong to the stream that the call runs on, so that the
    allocator reuses their memory in that stream's order.  A handle is taken for a stream
    of t's device."""
    device = t.device if isinstance(t, torch.Tensor) and t.is_cuda else None
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif device is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _current(t):
    """The handle of the current stream of t's device (one lookup, without the Stream
    object that torch.cuda.current_stream() builds)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _done(got):
    """What the binding answered: results, or the status of a call that failed."""
    if type(got) is int:
        _check(got)
    return got


def _empty(like, *shape, dtype):
    return torch.empty(shape, dtype=dtype, device=like.device)


def _scratch(like, nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None


def rowwise_int8(x, *, stream=None):
    """int8 codes of x's shape and one fp32 power-of-two scale per row.

    ``x`` is [rows, dim] fp32 or bf16 with dense rows."""
    if stream is not None:
        with _on(stream, x):
            return rowwise_int8(x)
    got = _qcbind.rowwise_int8(x)
    if got is not None:
        return _done(got)
    stride = _rows(x, "x", _CODE_OF)
    rows, dim = x.shape
    with _device_of(x=x):
        codes = _empty(x, rows, dim, dtype=torch.int8)
        scale = _empty(x, rows, dtype=torch.float32)
        _check(lib.qc_rowwise_int8(x.data_ptr(), _CODE_OF[x.dtype], stride, rows, dim, codes.data_ptr(),
                                   scale.data_ptr(), _current(x)))
    return codes, scale


def rowwise_int8_dequant(codes, row_scale, *, dtype=torch.bfloat16, stream=None):
    """The rows that the codes stand for."""
    if stream is not None:
        with _on(stream, codes):
            return rowwise_int8_dequant(codes, row_scale, dtype=dtype)
    code = _dtype(dtype)
    got = _qcbind.rowwise_int8_dequant(codes, row_scale, dtype is torch.bfloat16)
    if got is not None:
        return _done(got)
    _codes(codes, row_scale, "row")
    rows, dim = codes.shape
    with _device_of(codes=codes, row_scale=row_scale):
        out = _empty(codes, rows, dim, dtype=dtype)
        _check(lib.qc_rowwise_int8_dequant(codes.data_ptr(), row_scale.data_ptr(), rows, dim, out.data_ptr(), code, dim,
                                           _current(codes)))
    return out


def int8_matmul(x_codes, x_scale, w_codes, w_scale, bias=None, *, dtype=torch.bfloat16, stream=None):
    """y [T, N] from the codes of x [T, K] and of w [N, K], their scales, and an
    optional fp32 bias [N]."""
    if stream is not None:
        with _on(stream, x_codes):
            return int8_matmul(x_codes, x_scale, w_codes, w_scale, bias, dtype=dtype)
    code = _dtype(dtype)
    got = _qcbind.int8_matmul(x_codes, x_scale, w_codes, w_scale, bias, dtype is torch.bfloat16)
    if got is not None:
        return _done(got)
    _codes(x_codes, x_scale, "x")
    _codes(w_codes, w_scale, "w")
    if bias is not None:
        _dense(bias, "bias", _F32, (w_codes.shape[0],))
    if w_codes.shape[1] != x_codes.shape[1]:
        raise ValueError(f"w_codes has rows of {w_codes.shape[1]}, x_codes of {x_codes.shape[1]}")
    T, K = x_codes.shape
    N = w_codes.shape[0]
    with _device_of(x_codes=x_codes, x_scale=x_scale, w_codes=w_codes, w_scale=w_scale, bias=bias):
        y = _empty(x_codes, T, N, dtype=dtype)
        nbytes = lib.qc_int8_matmul_codes_workspace(x_codes.data_ptr(), w_codes.data_ptr(), T, N, K)
        ws = _scratch(x_codes, nbytes)
        _check(lib.qc_int8_matmul(x_codes.data_ptr(), x_scale.data_ptr(), w_codes.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                                  T, N, K, y.data_ptr(), code, N, _ptr(ws), nbytes, _current(x_codes)))
    return y


def int8_input_grad(dy, w_codes, w_scale, *, dtype=torch.bfloat16, stream=None):
    """dx [T, K] from dy [T, N] bf16 (dense rows) and the codes of w [N, K].

    The decoded weights are multiplied as bf16, which is exact under the powers of two of
    rowwise_int8; under any other w_scale each is rounded once (2^-9), which the forward
    product, whose scales are applied to its sums, does not do."""
    if stream is not None:
        with _on(stream, dy):
            return int8_input_grad(dy, w_codes, w_scale, dtype=dtype)
    code = _dtype(dtype)
    got = _qcbind.int8_input_grad(dy, w_codes, w_scale, dtype is torch.bfloat16)
    if got is not None:
        return _done(got)
    _codes(w_codes, w_scale, "w")
    stride = _rows(dy, "dy", _BF16)
    T, n = dy.shape
    N, K = w_codes.shape
    if n != N:
        raise ValueError(f"dy has rows of {n}, w_codes has {N} rows")
    with _device_of(dy=dy, w_codes=w_codes, w_scale=w_scale):
        dx = _empty(dy, T, K, dtype=dtype)
        nbytes = lib.qc_int8_input_grad_workspace(T, N, K)
        ws = _scratch(dy, nbytes)
        _check(lib.qc_int8_input_grad(dy.data_ptr(), stride, w_codes.data_ptr(), w_scale.data_ptr(), T, N, K,
                                      dx.data_ptr(), code, K, _ptr(ws), nbytes, _current(dy)))
    return dx


def int8_weight_grad(dy, x_codes, x_scale, *, dtype=torch.float32, with_bias=False, into=None,
                     stream=None):
    """(dw [N, K], dbias [N] fp32 or None) from dy [T, N] bf16 (dense rows) and the
    codes of x [T, K]; the decoded x is a bf16, as in int8_input_grad.  ``into`` = (dw, dbias or None), fp32: the gradients are
    added to them and they are returned; ``dtype`` and ``with_bias`` then say nothing and are
    refused where they contradict it."""
    if stream is not None:
        with _on(stream, dy):
            return int8_weight_grad(dy, x_codes, x_scale, dtype=dtype, with_bias=with_bias, into=into)
    if into is None:
        _dtype(dtype)
        got = _qcbind.int8_weight_grad(dy, x_codes, x_scale, dtype is torch.bfloat16, bool(with_bias))
        if got is not None:
            return _done(got)
    _codes(x_codes, x_scale, "x")
    stride = _rows(dy, "dy", _BF16)
    T, K = x_codes.shape
    t, N = dy.shape
    if t != T:
        raise ValueError(f"dy has {t} rows, x_codes {T}")
    dw = dbias = None
    if into is not None:
        dw, dbias = into
        if dtype is not torch.float32:
            raise ValueError(f"into takes fp32 gradients, and dtype is {dtype}")
        if with_bias and dbias is None:
            raise ValueError("with_bias, but into holds no dbias")
        _dense(dw, "dw", _F32, (N, K))
        if dbias is not None:
            _dense(dbias, "dbias", _F32, (N,))
    with _device_of(dy=dy, x_codes=x_codes, x_scale=x_scale, dw=dw, dbias=dbias):
        if into is None:
            dw = _empty(dy, N, K, dtype=dtype)
            dbias = _empty(dy, N, dtype=torch.float32) if with_bias else None
        nbytes = lib.qc_int8_weight_grad_workspace(T, N, K)
        ws = _scratch(dy, nbytes)
        _check(lib.qc_int8_weight_grad(dy.data_ptr(), stride, x_codes.data_ptr(), x_scale.data_ptr(), T, N, K,
                                       dw.data_ptr(), _CODE_OF[dtype], _ptr(dbias),
                                       0 if into is None else QC_ACCUMULATE_INTO_OUT, _ptr(ws), nbytes,
                                       _current(dy)))
    return dw, dbias


def swiglu_encode(gate_up, *, stream=None):
    """(h_codes [T, F], h_scale [T], saved_codes [T, 2F], saved_scale [T, 2]) of
    gate_up [T, 2F], a row's F gates followed by its F ups (dense rows, fp32 or bf16)."""
    if stream is not None:
        with _on(stream, gate_up):
            return swiglu_encode(gate_up)
    got = _qcbind.swiglu_encode(gate_up)
    if got is not None:
        return _done(got)
    stride = _rows(gate_up, "gate_up", _CODE_OF)
    rows, two = gate_up.shape
    if two % 2:
        raise ValueError(f"gate_up has rows of {two}; an even number is needed")
    with _device_of(gate_up=gate_up):
        h_codes = _empty(gate_up, rows, two // 2, dtype=torch.int8)
        h_scale = _empty(gate_up, rows, dtype=torch.float32)
        saved_codes = _empty(gate_up, rows, two, dtype=torch.int8)
        saved_scale = _empty(gate_up, rows, 2, dtype=torch.float32)
        _check(lib.qc_swiglu_encode(gate_up.data_ptr(), _CODE_OF[gate_up.dtype], stride, rows, two // 2,
                                    h_codes.data_ptr(), h_scale.data_ptr(), saved_codes.data_ptr(),
                                    saved_scale.data_ptr(), _current(gate_up)))
    return h_codes, h_scale, saved_codes, saved_scale


def swiglu_backward(dh, saved_codes, saved_scale, *, stream=None):
    """dgate_up [T, 2F] of dh's type from dh [T, F] (dense rows, fp32 or bf16) and
    what swiglu_encode saved."""
    if stream is not None:
        with _on(stream, dh):
            return swiglu_backward(dh, saved_codes, saved_scale)
    got = _qcbind.swiglu_backward(dh, saved_codes, saved_scale)
    if got is not None:
        return _done(got)
    stride = _rows(dh, "dh", _CODE_OF)
    rows, dim = dh.shape
    _dense(saved_codes, "saved_codes", _I8, (rows, 2 * dim))
    _dense(saved_scale, "saved_scale", _F32, (rows, 2))
    with _device_of(dh=dh, saved_codes=saved_codes, saved_scale=saved_scale):
        out = _empty(dh, rows, 2 * dim, dtype=dh.dtype)
        _check(lib.qc_swiglu_backward(dh.data_ptr(), _CODE_OF[dh.dtype], stride, saved_codes.data_ptr(),
                                      saved_scale.data_ptr(), rows, dim, out.data_ptr(), 2 * dim, _current(dh)))
    return out
