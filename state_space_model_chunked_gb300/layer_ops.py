"""ctypes binding of the layer's steps around the scan: the RMS norm with the
residual's addition, the matrix product with its epilogue and the gated linear
recurrence (argument marshalling only; contracts in include/ssd.h).

Matrices may be column ranges of wider ones: unit-stride columns, and leading
dimensions that lie at one row stride.  Outputs, and workspaces that are not
given, are allocated with torch on the inputs' device; every call runs on the
current stream of that device.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from ._binding import FP8_E4M3, SsdError, _check, _host_offsets, lib_path, load

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2, "relu": 3}
GATED_SCAN_CHECKPOINT = 64      # tokens between the states kept for gated_scan_bwd
_CODES = {torch.float32: 0, torch.bfloat16: 1, FP8_E4M3: 2}
_F32 = torch.float32
_BAD = ctypes.c_size_t(-1).value
_INT_MAX = 2 ** 31 - 1


_marshal_module = None


def _marshal():
    """The compiled marshalling of plain calls (ssd_marshal.so, beside
    libssd.so).  Its functions answer plain calls and return None for others; a
    status that is not OK comes back as an int."""
    global _marshal_module
    if _marshal_module is None:
        load()
        path = os.path.join(os.path.dirname(lib_path()), "ssd_marshal.so")
        if not os.path.exists(path):
            raise ImportError(f"ssd_marshal.so not found at {path}; build it with "
                              "`python -m state_space_model_chunked_gb300.build`")
        spec = importlib.util.spec_from_file_location("ssd_marshal", path)
        _marshal_module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(_marshal_module)
    return _marshal_module


def _plain(fn, answer):
    """A marshalled call's answer, an error status raised."""
    if answer.__class__ is int:
        _check(fn, answer)
    return answer


def _code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float8_e4m3fn, got {dtype}")
    return code


def _activation(name):
    code = ACTIVATIONS.get("none" if name is None else name)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}")
    return code


# The checks below are one expression a tensor on the way that passes: a call of
# one token is as long as its marshalling.
def _cuda(t, name):
    """The tensor's device index."""
    if t is None:
        raise ValueError(f"{name} is required")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() and t.shape[-1] > _INT_MAX:
        raise ValueError(f"{name} has {t.shape[-1]} columns, more than a C int holds")
    return index


def _refuse(t, name, dtype, index, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _full(t, name, dtype, index, shape):
    """Address of a contiguous array (None: no array)."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.get_device() != index or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, dtype, index, shape)
    return t.data_ptr()


def _out(t, name, dtype, index, device, shape):
    """(array, address) of an output: the caller's, or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _full(t, name, dtype, index, shape)


def _row_stride(t, name):
    """Distance of two rows of a matrix whose leading dimensions lie at one stride."""
    if t.dim() < 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected at least two dimensions")
    width = t.shape[-1]
    if t.is_contiguous():
        return width
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit-stride columns, got strides {t.stride()}")
    row, step = None, None
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if row is None:
            row = stride
        elif stride != step:
            raise ValueError(f"{name}: rows do not lie at one stride (shape {tuple(t.shape)}, "
                             f"strides {t.stride()})")
        step = stride * size
    row = width if row is None else row
    if row < width:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return row


def _rows(t, name, dtype, index, shape):
    """(address, row stride) of a matrix (None: no matrix)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _refuse(t, name, dtype, index, shape)
    if t.is_contiguous() and t.dim() > 1:
        return t.data_ptr(), shape[-1]
    return t.data_ptr(), _row_stride(t, name)


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _call(index, fn, *args):
    """The C call on the device's current stream; `args` without the stream."""
    if index == _current_device():
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _check(fn.__name__, rc)


def _size(index, fn, *args):
    if index == _current_device():
        n = fn(*args)
    else:
        with torch.cuda.device(index):
            n = fn(*args)
    if n == _BAD:
        raise SsdError(fn.__name__, 1, "invalid sizes")
    return n


def _index(device):
    if device is None:
        return torch.cuda.current_device()
    device = torch.device(device)
    return torch.cuda.current_device() if device.index is None else device.index


def _scratch(workspace, need, device):
    """(tensor or None, address, bytes) of a call's workspace."""
    if need == 0:
        return None, None, 0
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _count(shape):
    n = 1
    for v in shape:
        n *= v
    return n


# ----------------------------------------------------------------------- norm
def rmsnorm_fwd(x, weight, residual=None, *, eps=1e-5, out_dtype=None, y=None, residual_out=None,
                rstd=None, scale=None):
    """RMS norm of s = x + residual over the last dimension:
    y = s * rsqrt(mean(s^2) + eps) * weight.

    x [..., width] f32 or bf16; residual (x's shape; x's dtype or f32) or
    None; weight [width] f32; out_dtype f32, bf16 (default: x's) or
    float8_e4m3fn, with one scale a row (y * scale[..., None] is the value).
    Returns (y, residual_out = s in the residual's dtype or None, rstd [...]
    f32, scale [...] f32 or None).  residual_out may be the residual itself."""
    if x is not None and y is None and residual_out is None and rstd is None and scale is None:
        got = (_marshal_module or _marshal()).rmsnorm_fwd(
            x, weight, residual, eps, _code(x.dtype if out_dtype is None else out_dtype, "out_dtype"))
        if got is not None:
            return _plain("ssd_rmsnorm_fwd", got)
    lib = load()
    at, dev, dtype = _cuda(x, "x"), x.device, x.dtype
    shape = x.shape
    rows_shape, width = shape[:-1], shape[-1]
    out_dtype = dtype if out_dtype is None else out_dtype
    xc, oc = _code(dtype, "x"), _code(out_dtype, "out_dtype")
    xp, xs = _rows(x, "x", dtype, at, shape)
    if residual is not None:
        stream = residual.dtype
        rp, rs = _rows(residual, "residual", stream, at, shape)
        sc = _code(stream, "residual")
        residual_out, sp = _out(residual_out, "residual_out", stream, at, dev, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    else:
        rp, rs, sc, sp = None, 0, xc, None
    y, yp = _out(y, "y", out_dtype, at, dev, shape)
    rstd, tp = _out(rstd, "rstd", _F32, at, dev, rows_shape)
    if out_dtype is FP8_E4M3:
        scale, cp = _out(scale, "scale", _F32, at, dev, rows_shape)
    else:
        scale, cp = None, None
    _call(at, lib.ssd_rmsnorm_fwd, xp, rp, _full(weight, "weight", _F32, at, (width,)), eps, xc,
          sc, oc, _count(rows_shape), width, xs, rs, yp, sp, tp, cp)
    return y, residual_out, rstd, scale


def rmsnorm_bwd_workspace_bytes(rows, width, device=None):
    """Workspace bytes of rmsnorm_bwd on the device."""
    return _size(_index(device), load().ssd_rmsnorm_bwd_workspace_bytes, rows, width)


def rmsnorm_bwd(dy, s, weight, rstd, dresidual=None, *, dx=None, ds=None, dweight=None,
                workspace=None):
    """Gradients of rmsnorm_fwd: dy [..., width] of y; s, rstd: its residual_out
    (or x) and rstd; dresidual (s's dtype): the gradient that reached
    residual_out from elsewhere.  Returns (dx, ds, dweight): the gradient of x
    in dy's dtype and of the residual in s's (one tensor when those agree),
    and of the weight, f32."""
    if dx is None and ds is None and dweight is None and workspace is None:
        got = (_marshal_module or _marshal()).rmsnorm_bwd(dy, s, weight, rstd, dresidual)
        if got is not None:
            return _plain("ssd_rmsnorm_bwd", got)[:3]
    lib = load()
    at, dev = _cuda(dy, "dy"), dy.device
    shape, width = dy.shape, dy.shape[-1]
    yc = _code(dy.dtype, "dy")
    yp, ys = dy.data_ptr(), _row_stride(dy, "dy")
    sp, ss = _rows(s, "s", s.dtype, at, shape)
    dp, dstride = _rows(dresidual, "dresidual", s.dtype, at, shape)
    rows = _count(shape[:-1])
    if dx is None:
        dx = torch.empty(shape, dtype=dy.dtype, device=dev)
    one = s.dtype == dy.dtype
    if one:
        if ds is not None and ds is not dx:
            raise ValueError("ds is dx when dy and s have one dtype")
    elif ds is None:
        ds = torch.empty(shape, dtype=s.dtype, device=dev)
    if dweight is None:
        dweight = torch.empty((width,), dtype=_F32, device=dev)
    need = _size(at, lib.ssd_rmsnorm_bwd_workspace_bytes, rows, width)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_rmsnorm_bwd, yp, sp, _full(weight, "weight", _F32, at, (width,)),
          _full(rstd, "rstd", _F32, at, shape[:-1]), dp, yc, _code(s.dtype, "s"), rows, width, ys,
          ss, dstride, _full(dx, "dx", dy.dtype, at, shape),
          None if one else _full(ds, "ds", s.dtype, at, shape),
          _full(dweight, "dweight", _F32, at, (width,)), wp, wb)
    return dx, dx if one else ds, dweight


# -------------------------------------------------------------------- product
def linear_bwd_workspace_bytes(dtype, tokens, features, inner, activation=None, device=None):
    """Workspace bytes of linear_bwd on the device."""
    return _size(_index(device), load().ssd_linear_bwd_workspace_bytes, _code(dtype, "dtype"),
                 _activation(activation), tokens, features, inner)


PRODUCTS = {"forward": 0, "dx": 1, "dw": 2, "gradients": 3}
PATHS = ("fp32", "fp32_few", "few", "few_split", "whole", "pairs", "split", "split_pairs",
         "pairs_and_split", "together", "apart")


def linear_path(dtype, tokens, features, inner, product="forward", device=None):
    """The kernel (one of PATHS, see ssd_path in include/ssd.h) that linear_fwd takes for
    these sizes on the device, or linear_bwd for its product "dx", "dw" or both
    ("gradients"), when the operands are contiguous and aligned."""
    if product not in PRODUCTS:
        raise ValueError(f"product must be one of {', '.join(PRODUCTS)}, got {product!r}")
    fn, code, index = load().ssd_linear_path, _code(dtype, "dtype"), _index(device)
    with torch.cuda.device(index):
        path = fn(PRODUCTS[product], code, tokens, features, inner)
    if path < 0:
        raise SsdError(fn.__name__, 1, "invalid sizes")
    return PATHS[path]


def linear_fwd(x, w, bias=None, residual=None, *, activation=None, x_scale=None, w_scale=None,
               out_dtype=None, y=None, preact=None, return_preact=False):
    """y = act(x w^T * x_scale[:, None] * w_scale + bias) + residual.

    x [..., inner] and w [features, inner]: f32, bf16, or float8_e4m3fn with
    x_scale [...] and w_scale [features] f32.  bias [features] f32; residual
    [..., features] in out_dtype (default bf16 for bf16 and fp8 inputs, f32
    for f32 ones); activation None, "silu", "gelu" or "relu".  y may be the
    residual itself.  Returns y, or (y, preact) with return_preact: the values
    before the activation, which linear_bwd needs."""
    act = _activation(activation)
    if x is not None and y is None and preact is None and not return_preact:
        out = out_dtype or (_F32 if x.dtype is _F32 else torch.bfloat16)
        got = (_marshal_module or _marshal()).linear_fwd(x, w, bias, residual, act, x_scale, w_scale,
                                                         _code(out, "out_dtype"))
        if got is not None:
            return _plain("ssd_linear_fwd", got)
    lib = load()
    at, dev = _cuda(x, "x"), x.device
    xc = _code(x.dtype, "x")
    lead, inner = x.shape[:-1], x.shape[-1]
    if w is None or w.dim() != 2 or w.shape[0] > _INT_MAX:
        raise ValueError("w must be [features, inner]")
    features = w.shape[0]
    xp, xs = x.data_ptr(), _row_stride(x, "x")
    kept = _F32 if xc == 0 else torch.bfloat16
    out_dtype = kept if out_dtype is None else out_dtype
    oc = _code(out_dtype, "out_dtype")
    shape = lead + (features,)
    rp, rs = _rows(residual, "residual", out_dtype, at, shape)
    if y is None:
        y = torch.empty(shape, dtype=out_dtype, device=dev)
        yp, ys = y.data_ptr(), features
    else:
        yp, ys = _rows(y, "y", out_dtype, at, shape)
    if return_preact and preact is None:
        preact = torch.empty(shape, dtype=kept, device=dev)
    tokens = _count(lead)
    _call(at, lib.ssd_linear_fwd, xp, _full(x_scale, "x_scale", _F32, at, lead),
          _full(w, "w", x.dtype, at, (features, inner)),
          _full(w_scale, "w_scale", _F32, at, (features,)),
          _full(bias, "bias", _F32, at, (features,)), rp, act, xc, oc, tokens, features, inner,
          xs, rs, yp, ys, _full(preact, "preact", kept, at, shape))
    return (y, preact) if return_preact else y


def linear_bwd(dy, x, w, preact=None, *, activation=None, bias=True, need_dx=True, need_dw=True,
               dx=None, dw=None, dbias=None, workspace=None):
    """Gradients of linear_fwd (f32 or bf16): dy [..., features]; x and w as
    given to it; preact as it returned (with an activation).  Returns
    (dx, dw, dbias): in dy's dtype, dy's dtype and f32; None for what is not
    wanted (need_dx, need_dw, bias).  The residual's gradient is dy."""
    act = _activation(activation)
    if need_dx and need_dw and dx is None and dw is None and dbias is None and workspace is None:
        got = (_marshal_module or _marshal()).linear_bwd(dy, x, w, preact, act, bias)
        if got is not None:
            return _plain("ssd_linear_bwd", got)[:3]
    lib = load()
    at, dev = _cuda(dy, "dy"), dy.device
    dt, code = dy.dtype, _code(dy.dtype, "dy")
    lead, features = dy.shape[:-1], dy.shape[-1]
    inner = x.shape[-1]
    yp, ys = dy.data_ptr(), _row_stride(dy, "dy")
    xp, xs = _rows(x, "x", dt, at, lead + (inner,))
    tokens = _count(lead)
    if need_dx and dx is None:
        dx = torch.empty(lead + (inner,), dtype=dt, device=dev)
    if need_dw and dw is None:
        dw = torch.empty((features, inner), dtype=dt, device=dev)
    if bias and dbias is None:
        dbias = torch.empty((features,), dtype=_F32, device=dev)
    need = _size(at, lib.ssd_linear_bwd_workspace_bytes, code, act, tokens, features, inner)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_linear_bwd, yp, xp, _full(w, "w", dt, at, (features, inner)),
          _full(preact, "preact", dt, at, dy.shape), act, code, tokens, features, inner, ys, xs,
          _full(dx, "dx", dt, at, lead + (inner,)), _full(dw, "dw", dt, at, (features, inner)),
          _full(dbias, "dbias", _F32, at, (features,)), wp, wb)
    return dx, dw, dbias


# ----------------------------------------------------------------- recurrence
def gated_scan_workspace_bytes(dtype, tokens, width, device=None):
    """Workspace bytes of gated_scan_fwd and gated_scan_bwd on the device."""
    return _size(_index(device), load().ssd_gated_scan_workspace_bytes, _code(dtype, "dtype"), tokens, width)


def _sequences(x, name, cu_seqlens, cu_seqlens_dev):
    """(nseq, length, host offsets' address, device offsets' address, tokens,
    what to keep alive) of x [b, L, width], or [T, width] with offsets."""
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [batch, length, width] "
                             "(or [tokens, width] with cu_seqlens)")
        return x.shape[0], x.shape[1], None, None, x.shape[0] * x.shape[1], None
    if x.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [tokens, width]")
    cu, cu_ptr = _host_offsets(cu_seqlens)
    if int(cu[-1]) != x.shape[0]:
        raise ValueError(f"cu_seqlens ends at {int(cu[-1])}, {name} holds {x.shape[0]} tokens")
    if cu_seqlens_dev is None:
        cu_seqlens_dev = torch.from_numpy(cu).to(x.device)
    dev_ptr = _full(cu_seqlens_dev, "cu_seqlens_dev", torch.int32, x.get_device(), (cu.size,))
    return cu.size - 1, 0, cu_ptr, dev_ptr, x.shape[0], (cu, cu_seqlens_dev)


def gated_scan_fwd(x, g, z=None, init_state=None, *, cu_seqlens=None, cu_seqlens_dev=None, y=None,
                   final_state=None, return_final=True, checkpoints=None, return_checkpoints=False,
                   workspace=None):
    """Gated linear recurrence h_t = f_t h_{t-1} + (1 - f_t) x_t, f = sigmoid(g),
    y = h (times silu(z) when z is given), for every channel by itself.

    x, g, z [batch, length, width] f32 or bf16; or [tokens, width] with
    cu_seqlens (and cu_seqlens_dev, which saves its copy) as in
    scan_fwd_varlen.  init_state [nseq, width] f32 or None.  Returns
    (y, final_state [nseq, width] f32 or None), and the states
    [ceil(tokens / 64), width] f32 that gated_scan_bwd needs with
    return_checkpoints.  Equal calls of more than 64 tokens may differ in their
    last fp32 bits: the order in which parts are joined follows their progress."""
    if (y is None and final_state is None and return_final and checkpoints is None
            and workspace is None):
        got = (_marshal_module or _marshal()).gated_scan_fwd(x, g, z, init_state, cu_seqlens,
                                                             cu_seqlens_dev, return_checkpoints)
        if got is not None:
            return _plain("ssd_gated_scan_fwd", got)[:3 if return_checkpoints else 2]
    lib = load()
    at, dev = _cuda(x, "x"), x.device
    code, shape, width = _code(x.dtype, "x"), x.shape, x.shape[-1]
    nseq, length, cu_ptr, cu_dev, tokens, _keep_cu = _sequences(x, "x", cu_seqlens, cu_seqlens_dev)
    xs = _row_stride(x, "x")
    gp, gs = _rows(g, "g", x.dtype, at, shape)
    zp, zs = _rows(z, "z", x.dtype, at, shape)
    if y is None:
        y = torch.empty(shape, dtype=x.dtype, device=dev)
    yp, ys = _rows(y, "y", x.dtype, at, shape)
    if final_state is None and return_final:
        final_state = torch.empty((nseq, width), dtype=_F32, device=dev)
    kept = (-(-tokens // GATED_SCAN_CHECKPOINT), width)
    if checkpoints is None and return_checkpoints:
        checkpoints = torch.empty(kept, dtype=_F32, device=dev)
    need = _size(at, lib.ssd_gated_scan_workspace_bytes, code, tokens, width)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_gated_scan_fwd, x.data_ptr(), gp, zp, code, nseq, length, cu_ptr, cu_dev,
          width, xs, gs, zs, _full(init_state, "init_state", _F32, at, (nseq, width)), yp, ys,
          _full(final_state, "final_state", _F32, at, (nseq, width)),
          _full(checkpoints, "checkpoints", _F32, at, kept), wp, wb)
    return (y, final_state, checkpoints) if return_checkpoints else (y, final_state)


def gated_scan_bwd(dy, x, g, checkpoints, z=None, init_state=None, dfinal=None, *, cu_seqlens=None,
                   cu_seqlens_dev=None, dx=None, dg=None, dz=None, dinit=None, return_dinit=True,
                   workspace=None):
    """Gradients of gated_scan_fwd: dy of y, dfinal [nseq, width] f32 of the
    final state (None: zeros); x, g, z, init_state and offsets as given to it
    and the checkpoints it returned.  dx, dg and dz may be column ranges of one
    matrix.  Returns (dx, dg, dz or None, dinit [nseq, width] f32 or None)."""
    if (dx is None and dg is None and dz is None and dinit is None and return_dinit
            and workspace is None):
        got = (_marshal_module or _marshal()).gated_scan_bwd(dy, x, g, checkpoints, z, init_state,
                                                             dfinal, cu_seqlens, cu_seqlens_dev)
        if got is not None:
            return _plain("ssd_gated_scan_bwd", got)
    lib = load()
    at, dev = _cuda(x, "x"), x.device
    code, shape, width = _code(x.dtype, "x"), x.shape, x.shape[-1]
    nseq, length, cu_ptr, cu_dev, tokens, _keep_cu = _sequences(x, "x", cu_seqlens, cu_seqlens_dev)
    xs = _row_stride(x, "x")
    yp, ys = _rows(dy, "dy", x.dtype, at, shape)
    gp, gs = _rows(g, "g", x.dtype, at, shape)
    zp, zs = _rows(z, "z", x.dtype, at, shape)
    if dx is None:
        dx = torch.empty(shape, dtype=x.dtype, device=dev)
    if dg is None:
        dg = torch.empty(shape, dtype=x.dtype, device=dev)
    if z is None:
        dz = None
    elif dz is None:
        dz = torch.empty(shape, dtype=x.dtype, device=dev)
    dxp, dxs = _rows(dx, "dx", x.dtype, at, shape)
    dgp, dgs = _rows(dg, "dg", x.dtype, at, shape)
    dzp, dzs = _rows(dz, "dz", x.dtype, at, shape)
    if dinit is None and return_dinit:
        dinit = torch.empty((nseq, width), dtype=_F32, device=dev)
    kept = (-(-tokens // GATED_SCAN_CHECKPOINT), width)
    if checkpoints is None:
        raise ValueError("checkpoints is required")
    need = _size(at, lib.ssd_gated_scan_workspace_bytes, code, tokens, width)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_gated_scan_bwd, yp, x.data_ptr(), gp, zp, code, nseq, length, cu_ptr, cu_dev,
          width, ys, xs, gs, zs, _full(init_state, "init_state", _F32, at, (nseq, width)),
          _full(checkpoints, "checkpoints", _F32, at, kept),
          _full(dfinal, "dfinal", _F32, at, (nseq, width)), dxp, dxs, dgp, dgs, dzp, dzs,
          _full(dinit, "dinit", _F32, at, (nseq, width)), wp, wb)
    return dx, dg, dz, dinit


def gated_state_update(state, x, g, z=None, *, y=None):
    """One token of the gated recurrence: state [..., width] f32, updated in
    place; x, g, z [..., width] f32 or bf16.  Returns y in x's dtype."""
    if y is None:
        got = (_marshal_module or _marshal()).gated_state_update(state, x, g, z)
        if got is not None:
            return _plain("ssd_gated_state_update", got)
    lib = load()
    at, dev = _cuda(x, "x"), x.device
    code, shape = _code(x.dtype, "x"), x.shape
    xs = _row_stride(x, "x")
    gp, gs = _rows(g, "g", x.dtype, at, shape)
    zp, zs = _rows(z, "z", x.dtype, at, shape)
    if state is None:
        raise ValueError("state is required")
    y, yp = _out(y, "y", x.dtype, at, dev, shape)
    _call(at, lib.ssd_gated_state_update, _full(state, "state", _F32, at, shape), x.data_ptr(),
          gp, zp, code, _count(shape[:-1]), shape[-1], xs, gs, zs, yp)
    return y
