"""ctypes binding of the gated delta rule: the recurrence over sequences, its
gradients and a single token (argument marshalling only; contracts in
include/ssd.h).

q, k, v and their gradients may be column ranges of wider matrices: a token's
values [groups, dstate] or [heads, headdim] contiguous, and the tokens at one
stride.  Outputs, and workspaces that are not given, are allocated with torch on
the inputs' device; every call runs on the current stream of that device.
"""
from __future__ import annotations

import torch

from . import layer_ops as _ops
from ._binding import ALGO_AUTO, ALGO_SIMT, ALGO_TCGEN05, load
from .layer_ops import (_call, _code, _count, _cuda, _full, _index, _out, _plain, _refuse,
                        _row_stride, _scratch, _sequences, _size)

DELTA_SCAN_CHECKPOINT = 64      # tokens between the states kept for delta_scan_bwd
_F32 = torch.float32


def _by_token(t, name, dtype, index, shape):
    """(address, stride of a token) of an array whose last two dimensions are a
    token's values."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _refuse(t, name, dtype, index, shape)
    width = shape[-2] * shape[-1]
    if t.is_contiguous():
        return t.data_ptr(), width
    if (shape[-1] > 1 and t.stride(-1) != 1) or (shape[-2] > 1 and t.stride(-2) != shape[-1]):
        raise ValueError(f"{name}: a token's values must be contiguous, got strides {t.stride()}")
    return t.data_ptr(), _row_stride(t.flatten(-2), name)


def _sizes(q, v, name="q"):
    """(device index, dtype code, lead, groups, dstate, heads, headdim)"""
    at = _cuda(q, name)
    _cuda(v, "v")
    if q.dim() < 3 or v.dim() != q.dim():
        raise ValueError(f"{name} and v have shapes {tuple(q.shape)} and {tuple(v.shape)}, expected "
                         "[..., groups, dstate] and [..., heads, headdim]")
    for t, what in ((q, name), (v, "v")):
        if t.shape[-2] > _ops._INT_MAX or 0 in t.shape[-2:]:
            raise ValueError(f"{what} has shape {tuple(t.shape)}")
    return at, _code(q.dtype, name), q.shape[:-2], q.shape[-2], q.shape[-1], v.shape[-2], v.shape[-1]


def _scale(scale, dstate):
    return dstate ** -0.5 if scale is None else scale


def _span(q, lead, cu_seqlens, cu_seqlens_dev):
    """_sequences of the tokens' axis."""
    if cu_seqlens is None and len(lead) != 2:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [batch, length, groups, dstate] "
                         "(or [tokens, groups, dstate] with cu_seqlens)")
    if cu_seqlens is not None and len(lead) != 1:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [tokens, groups, dstate]")
    return _sequences(q.select(-2, 0), "q", cu_seqlens, cu_seqlens_dev)


def delta_scan_checkpoints(tokens, nseq):
    """How many states delta_scan_fwd keeps places for (each [heads, headdim, dstate])."""
    return tokens // DELTA_SCAN_CHECKPOINT + nseq


def delta_scan_workspace_bytes(dtype, tokens, nseq, heads, headdim, dstate, groups, device=None,
                               algo=ALGO_AUTO):
    """Workspace bytes of delta_scan_fwd on the device."""
    return _size(_index(device), load().ssd_delta_scan_workspace_bytes_algo, algo,
                 _code(dtype, "dtype"), tokens, nseq, heads, headdim, dstate, groups)


def delta_scan_fwd(q, k, v, g, beta, init_state=None, *, scale=None, cu_seqlens=None,
                   cu_seqlens_dev=None, o=None, final_state=None, return_final=True,
                   checkpoints=None, return_checkpoints=False, workspace=None, algo=ALGO_AUTO):
    """Gated delta rule, for every head with its state S [headdim, dstate]:
    S' = exp(g_t) S_{t-1}, u_t = beta_t (v_t - S' k_t), S_t = S' + u_t k_t^T,
    o_t = scale S_t q_t (scale: dstate^-0.5 by default).

    q, k [batch, length, groups, dstate] and v [batch, length, heads, headdim] f32 or
    bf16; g (the decay's logarithm) and beta [batch, length, heads] f32; or [tokens,
    ...] with cu_seqlens (and cu_seqlens_dev) as in gated_scan_fwd.  heads is a
    multiple of groups.  init_state [nseq, heads, headdim, dstate] f32 or None.
    Returns (o in v's layout, final_state f32 or None), and with return_checkpoints
    the states [delta_scan_checkpoints(tokens, nseq), heads, headdim, dstate] f32
    that delta_scan_bwd needs.

    algo: ALGO_AUTO runs bf16 inputs on the tensor cores where sizes and alignments
    allow it, whose f32 results are 3e-6 to 6e-6 of their size off; ALGO_SIMT asks for
    f32 multiply-adds throughout (1e-7), token by token; ALGO_TCGEN05 refuses what the
    tensor cores do not take."""
    if (algo == ALGO_AUTO and o is None and final_state is None and checkpoints is None
            and workspace is None):
        got = (_ops._marshal_module or _ops._marshal()).delta_scan_fwd(
            q, k, v, g, beta, init_state, scale, cu_seqlens, cu_seqlens_dev, return_final,
            return_checkpoints)
        if got is not None:
            return _plain("ssd_delta_scan_fwd", got)[:3 if return_checkpoints else 2]
    lib = load()
    at, code, lead, groups, dstate, heads, headdim = _sizes(q, v)
    dev, dtype = q.device, q.dtype
    nseq, length, cu_ptr, cu_dev, tokens, _keep_cu = _span(q, lead, cu_seqlens, cu_seqlens_dev)
    qp, qs = _by_token(q, "q", dtype, at, q.shape)
    kp, ks = _by_token(k, "k", dtype, at, q.shape)
    vp, vs = _by_token(v, "v", dtype, at, lead + (heads, headdim))
    if o is None:
        o = torch.empty(v.shape, dtype=dtype, device=dev)
    op, os_ = _by_token(o, "o", dtype, at, v.shape)
    states = (nseq, heads, headdim, dstate)
    if final_state is None and return_final:
        final_state = torch.empty(states, dtype=_F32, device=dev)
    kept = (delta_scan_checkpoints(tokens, nseq),) + states[1:]
    if checkpoints is None and return_checkpoints:
        checkpoints = torch.empty(kept, dtype=_F32, device=dev)
    need = _size(at, lib.ssd_delta_scan_workspace_bytes_algo, algo, code, tokens, nseq, heads, headdim,
                 dstate, groups)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_delta_scan_fwd_algo, algo, qp, kp, vp, _full(g, "g", _F32, at, lead + (heads,)),
          _full(beta, "beta", _F32, at, lead + (heads,)), code, nseq, length, cu_ptr, cu_dev, heads,
          headdim, dstate, groups, qs, ks, vs, _scale(scale, dstate),
          _full(init_state, "init_state", _F32, at, states), op, os_,
          _full(final_state, "final_state", _F32, at, states),
          _full(checkpoints, "checkpoints", _F32, at, kept), wp, wb)
    return (o, final_state, checkpoints) if return_checkpoints else (o, final_state)


def delta_scan_bwd_workspace_bytes(dtype, tokens, nseq, heads, headdim, dstate, groups, device=None,
                                   algo=ALGO_AUTO):
    """Workspace bytes of delta_scan_bwd on the device (ALGO_AUTO: for whatever
    alignments)."""
    return _size(_index(device), load().ssd_delta_scan_bwd_workspace_bytes_algo, algo,
                 _code(dtype, "dtype"), tokens, nseq, heads, headdim, dstate, groups)


def delta_scan_bwd(do, q, k, v, g, beta, checkpoints, dfinal=None, *, scale=None, cu_seqlens=None,
                   cu_seqlens_dev=None, dq=None, dk=None, dv=None, dg=None, dbeta=None, dinit=None,
                   return_dinit=True, workspace=None, algo=ALGO_AUTO):
    """Gradients of delta_scan_fwd: do of o, dfinal [nseq, heads, headdim, dstate]
    f32 of the final state (None: zeros); q, k, v, g, beta, scale and offsets as
    given to it and the checkpoints it returned.  dq, dk and dv may be column ranges
    of one matrix.  algo as for delta_scan_fwd (the checkpoints may be of either).
    Returns (dq, dk, dv, dg, dbeta, dinit f32 or None)."""
    if (algo == ALGO_AUTO and dq is None and dk is None and dv is None and dg is None and dbeta is None and dinit is None
            and workspace is None):
        got = (_ops._marshal_module or _ops._marshal()).delta_scan_bwd(
            q, k, v, g, beta, dfinal, do, checkpoints, scale, cu_seqlens, cu_seqlens_dev, return_dinit)
        if got is not None:
            return _plain("ssd_delta_scan_bwd", got)
    lib = load()
    at, code, lead, groups, dstate, heads, headdim = _sizes(q, v)
    dev, dtype = q.device, q.dtype
    nseq, length, cu_ptr, cu_dev, tokens, _keep_cu = _span(q, lead, cu_seqlens, cu_seqlens_dev)
    values, gates = lead + (heads, headdim), lead + (heads,)
    dop, dos = _by_token(do, "do", dtype, at, values)
    qp, qs = _by_token(q, "q", dtype, at, q.shape)
    kp, ks = _by_token(k, "k", dtype, at, q.shape)
    vp, vs = _by_token(v, "v", dtype, at, values)
    dq = torch.empty(q.shape, dtype=dtype, device=dev) if dq is None else dq
    dk = torch.empty(q.shape, dtype=dtype, device=dev) if dk is None else dk
    dv = torch.empty(v.shape, dtype=dtype, device=dev) if dv is None else dv
    dqp, dqs = _by_token(dq, "dq", dtype, at, q.shape)
    dkp, dks = _by_token(dk, "dk", dtype, at, q.shape)
    dvp, dvs = _by_token(dv, "dv", dtype, at, values)
    dg, dgp = _out(dg, "dg", _F32, at, dev, gates)
    dbeta, dbp = _out(dbeta, "dbeta", _F32, at, dev, gates)
    states = (nseq, heads, headdim, dstate)
    if dinit is None and return_dinit:
        dinit = torch.empty(states, dtype=_F32, device=dev)
    if checkpoints is None:
        raise ValueError("checkpoints is required")
    kept = (delta_scan_checkpoints(tokens, nseq),) + states[1:]
    cp, fp, ip = (_full(checkpoints, "checkpoints", _F32, at, kept),
                  _full(dfinal, "dfinal", _F32, at, states), _full(dinit, "dinit", _F32, at, states))
    # the workspace of the kernels that run: where everything lies on 16 bytes the tensor cores'
    # (0: not for these sizes), else the others'
    sizes, need = (code, tokens, nseq, heads, headdim, dstate, groups), 0
    query = lib.ssd_delta_scan_bwd_workspace_bytes_algo
    where = dop | qp | kp | vp | cp | (fp or 0) | (ip or 0) | (dos | qs | ks | vs) * q.element_size()
    if algo != ALGO_SIMT and where % 16 == 0:
        need = _size(at, query, ALGO_TCGEN05, *sizes)
    if need == 0:
        need = _size(at, query, ALGO_SIMT, *sizes)
    _keep, wp, wb = _scratch(workspace, need, dev)
    _call(at, lib.ssd_delta_scan_bwd_algo, algo, dop, qp, kp, vp, _full(g, "g", _F32, at, gates),
          _full(beta, "beta", _F32, at, gates), code, nseq, length, cu_ptr, cu_dev, heads, headdim,
          dstate, groups, dos, qs, ks, vs, _scale(scale, dstate), cp, fp, dqp, dqs, dkp, dks, dvp,
          dvs, dgp, dbp, ip, wp, wb)
    return dq, dk, dv, dg, dbeta, dinit


def delta_state_update(state, q, k, v, g, beta, *, scale=None, o=None, state_out=None):
    """One token of the delta rule: state [batch, heads, headdim, dstate] f32 (or
    bf16 with bf16 inputs), q, k [batch, groups, dstate] and v [batch, heads, headdim]
    f32 or bf16, g and beta [batch, heads] f32.  The state is updated in place, or
    written to state_out with the old one left as it is.  Returns o in v's layout."""
    if o is None:
        got = (_ops._marshal_module or _ops._marshal()).delta_state_update(
            state, q, k, v, g, beta, scale, state_out)
        if got is not None:
            return _plain("ssd_delta_state_update", got)
    lib = load()
    at, code, lead, groups, dstate, heads, headdim = _sizes(q, v)
    if len(lead) != 1 or lead[0] > _ops._INT_MAX:
        raise ValueError(f"q has shape {tuple(q.shape)}, expected [batch, groups, dstate]")
    qp, qs = _by_token(q, "q", q.dtype, at, q.shape)
    kp, ks = _by_token(k, "k", q.dtype, at, q.shape)
    vp, vs = _by_token(v, "v", q.dtype, at, lead + (heads, headdim))
    _cuda(state, "state")
    sc, shape = _code(state.dtype, "state"), lead + (heads, headdim, dstate)
    sp = _full(state, "state", state.dtype, at, shape)
    np_ = sp if state_out is None else _full(state_out, "state_out", state.dtype, at, shape)
    o, op = _out(o, "o", q.dtype, at, q.device, v.shape)
    _call(at, lib.ssd_delta_state_update, sp, sc, np_, qp, kp, vp,
          _full(g, "g", _F32, at, lead + (heads,)), _full(beta, "beta", _F32, at, lead + (heads,)),
          code, _count(lead), heads, headdim, dstate, groups, qs, ks, vs, _scale(scale, dstate), op)
    return o
