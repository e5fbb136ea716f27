"""Operators of the parameters without Kronecker factors: root-mean-square norms and the token
embedding, forward and backward, with the diagonal factors that Kfac.diag_step takes; weight
matrices stepped along their orthogonalised momentum.

Argument marshalling only, in the manner of _block.py: outputs and workspaces may be given or are
allocated with torch; ValueError for a wrong shape, type or device, KfacError for what the library
refuses; ``stream`` as there; outside torch's autograd.  Definitions: include/kfac.h.
"""
from __future__ import annotations

import ctypes

import torch

from ._block import _call, _check, _device, _dtype, _elsewhere, _empty
from ._lib import (LIB, KFAC_BF16, KFAC_ORTHO_FULL, KFAC_ORTHO_HALF, NORM_DESC, NORM_GRAD_DESC,
                   EMBEDDING_DESC, ORTHO_DESC, ORTHO_STEP)


_cuda = {}   # devices by index: making one costs as much as two checks


def _new(shape, dtype, dev, stream):
    if stream is None:
        device = _cuda.get(dev)
        if device is None:
            device = _cuda[dev] = torch.device("cuda", dev)
        return torch.empty(shape, dtype=dtype, device=device)
    return _empty(shape, dtype, dev, stream)


def _like(t, shape, dtype, dev, stream):
    """A contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if stream is None and t.is_contiguous() else _new(shape, dtype, dev, stream)


def _sized(f, what, dev, *args):
    """The bytes that f(*args, &bytes) gives on the tensors' device."""
    n = ctypes.c_size_t(0)
    with torch.cuda.device(dev):   # the plan may depend on the device's SM count
        _check(f(*args, ctypes.byref(n)), what)
    return n.value


def _kept(nbytes, dev):
    """A workspace tensor to be kept by the caller."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", dev))


def _workspace(what, workspace, nbytes, dev, stream):
    """A call's workspace: the caller's, or its own."""
    if workspace is None:
        return _new((max(nbytes, 256),), torch.uint8, dev, stream)
    if workspace.get_device() != dev:
        _elsewhere(what, "workspace", workspace, dev)
    if not workspace.is_contiguous():
        raise ValueError(f"{what}: workspace is contiguous")
    return workspace


# ------------------------------------------------------------------------------------- norms

def _ld(what, name, t, shape, dtype, dev):
    """Leading dimension of t [..., cols]: contiguous, or 2-D with contiguous rows."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return shape[-1]
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what}: {name} is {t.dtype} {tuple(t.shape)}, not {dtype} {tuple(shape)}")
    if t.get_device() != dev:
        _elsewhere(what, name, t, dev)
    if t.dim() != 2 or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{what}: {name} is contiguous, or 2-D with contiguous rows")
    return t.stride(0)


def _vector(what, name, t, n, dev):
    """Address of a contiguous float32 [n] tensor (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: {name} is float32 [{n}], contiguous")
    if t.get_device() != dev:
        _elsewhere(what, name, t, dev)
    return t.data_ptr()


def _statistics(what, name, t, shape, dev):
    """Address of a contiguous float32 tensor of this shape."""
    if t.dtype is not torch.float32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: {name} is float32 {tuple(shape)}, contiguous")
    if t.get_device() != dev:
        _elsewhere(what, name, t, dev)
    return t.data_ptr()


def _channels(what, name, t):
    """(kfac_dtype, device, shape, rows, channels) of t [..., channels]."""
    dt, dev, shape = _dtype(t, what), _device(t, what), t.shape
    if not shape:
        raise ValueError(f"{what}: {name} is [..., channels]")
    cols = shape[-1]
    return dt, dev, shape, t.numel() // cols if cols else 0, cols


def rms_norm(x, gain=None, residual=None, eps: float = 1e-6, out=None, residual_out=None,
             rstd=None, stream=None):
    """kfac_rms_norm: the root-mean-square norm of x + residual, times gain (float32 [channels]);
    returns (out, residual_out, rstd).  x: [..., channels], contiguous, or 2-D with contiguous
    rows.  residual_out = x + residual (None without a residual); it may be x or residual.  The
    backward pass takes it (x without a residual) and rstd, float32 [...]."""
    what = "rms_norm"
    dt, dev, shape, rows, cols = _channels(what, "x", x)
    dtype = x.dtype
    ldx = _ld(what, "x", x, shape, dtype, dev)
    ldr = ldh = 0
    rp = hp = None
    if residual is not None:
        ldr, rp = _ld(what, "residual", residual, shape, dtype, dev), residual.data_ptr()
        if residual_out is None:
            residual_out, ldh = _like(x, shape, dtype, dev, stream), cols
            hp = residual_out.data_ptr()
    if residual_out is not None and hp is None:
        ldh, hp = _ld(what, "residual_out", residual_out, shape, dtype, dev), residual_out.data_ptr()
    if out is None:
        out, ldy = _like(x, shape, dtype, dev, stream), cols
    else:
        ldy = _ld(what, "out", out, shape, dtype, dev)
    if rstd is None:
        rstd = _new(shape[:-1], torch.float32, dev, stream)
        sp = rstd.data_ptr()
    else:
        sp = _statistics(what, "rstd", rstd, shape[:-1], dev)
    _call(LIB.kfac_rms_norm, "kfac_rms_norm", dev, stream,
          NORM_DESC.pack(dt, rows, cols, eps, ldx, ldr, ldh, ldy, 0, 0), x.data_ptr(), rp,
          _vector(what, "gain", gain, cols, dev), hp, out.data_ptr(), sp, None, None)
    return out, residual_out, rstd


def rms_norm_e4m3(x, gain=None, residual=None, eps: float = 1e-6, group: int = 0, out=None,
                  scales=None, residual_out=None, stream=None):
    """kfac_rms_norm with its result in 8 bits: (out float8_e4m3fn, scales float32 [..., groups],
    residual_out); out * scale of its group is the norm.  group: 32, 64 or 128 channels per scale, or
    0 for one per row."""
    what = "rms_norm_e4m3"
    dt, dev, shape, rows, cols = _channels(what, "x", x)
    dtype = x.dtype
    if group not in (0, 32, 64, 128):
        raise ValueError(f"{what}: group is 32, 64 or 128 channels, or 0 for the whole row")
    ldx = _ld(what, "x", x, shape, dtype, dev)
    ldr = ldh = 0
    rp = hp = None
    if residual is not None:
        ldr, rp = _ld(what, "residual", residual, shape, dtype, dev), residual.data_ptr()
        if residual_out is None:
            residual_out = _new(shape, dtype, dev, stream)
    if residual_out is not None:
        ldh, hp = _ld(what, "residual_out", residual_out, shape, dtype, dev), residual_out.data_ptr()
    if out is None:
        out, ldq = _new(shape, torch.float8_e4m3fn, dev, stream), cols
    else:
        ldq = _ld(what, "out", out, shape, torch.float8_e4m3fn, dev)
    groups = (*shape[:-1], -(-cols // group) if group else 1)
    if scales is None:
        scales = _new(groups, torch.float32, dev, stream)
        sp = scales.data_ptr()
    else:
        sp = _statistics(what, "scales", scales, groups, dev)
    _call(LIB.kfac_rms_norm, "kfac_rms_norm", dev, stream,
          NORM_DESC.pack(dt, rows, cols, eps, ldx, ldr, ldh, 0, ldq, group), x.data_ptr(), rp,
          _vector(what, "gain", gain, cols, dev), hp, None, None, out.data_ptr(), sp)
    return out, scales, residual_out


def rms_norm_workspace(x):
    """A workspace tensor for rms_norm_backward of tensors like x, to be kept and passed to it."""
    _, dev, _, rows, cols = _channels("rms_norm_workspace", "x", x)
    return _kept(_sized(LIB.kfac_rms_norm_workspace_size, "kfac_rms_norm_workspace_size", dev, rows, cols), dev)


def rms_norm_backward(dout, x, gain, rstd, dresidual=None, dx=None, dgain=None, dgain_square=None,
                      square: bool = False, workspace=None, stream=None):
    """kfac_rms_norm_backward: (dx, dgain, dgain_square) for the gradient dout of rms_norm's out.
    x: its residual_out (its x without a residual); dresidual: the gradient of residual_out from
    its other readers, added to dx, which is the gradient of x and of residual.  dgain_square
    (square=True, or a tensor given): the mean over the rows of the gain's squared gradient, which
    Kfac.diag_step takes as g_new; otherwise None."""
    what = "rms_norm_backward"
    dt, dev, shape, rows, cols = _channels(what, "dout", dout)
    dtype = dout.dtype
    lddy = _ld(what, "dout", dout, shape, dtype, dev)
    ldh = _ld(what, "x", x, shape, dtype, dev)
    lddh, dhp = 0, None
    if dresidual is not None:
        lddh, dhp = _ld(what, "dresidual", dresidual, shape, dtype, dev), dresidual.data_ptr()
    sp = _statistics(what, "rstd", rstd, shape[:-1], dev)
    if dx is None:
        dx, lddx = _like(dout, shape, dtype, dev, stream), cols
    else:
        lddx = _ld(what, "dx", dx, shape, dtype, dev)
    if dgain is None:
        dgain = _new((cols,), torch.float32, dev, stream)
        gp = dgain.data_ptr()
    else:
        gp = _vector(what, "dgain", dgain, cols, dev)
    if dgain_square is None and square:
        dgain_square = _new((cols,), torch.float32, dev, stream)
    workspace = _workspace(what, workspace, 0 if workspace is not None else _sized(
        LIB.kfac_rms_norm_workspace_size, "kfac_rms_norm_workspace_size", dev, rows, cols), dev, stream)
    _call(LIB.kfac_rms_norm_backward, "kfac_rms_norm_backward", dev, stream,
          NORM_GRAD_DESC.pack(dt, rows, cols, lddy, ldh, lddh, lddx), dout.data_ptr(), x.data_ptr(),
          _vector(what, "gain", gain, cols, dev), sp, dhp, dx.data_ptr(), gp,
          _vector(what, "dgain_square", dgain_square, cols, dev), workspace.data_ptr(),
          workspace.nbytes)
    return dx, dgain, dgain_square


# --------------------------------------------------------------------------------- embedding

_ID_BITS = {torch.int32: 32, torch.int64: 64}


def _ids(what, ids, dev):
    bits = _ID_BITS.get(ids.dtype)
    if bits is None or not ids.is_contiguous():
        raise ValueError(f"{what}: ids are int32 or int64, contiguous, not {ids.dtype}")
    if ids.get_device() != dev:
        _elsewhere(what, "ids", ids, dev)
    return bits


def embedding(ids, table, scale: float = 1.0, out=None, stream=None):
    """kfac_embedding: out [..., width] = scale * table[ids] for ids int32 or int64 [...]; the row of
    an id outside the table is NaN.  table: [rows, width], rows contiguous."""
    what = "embedding"
    dt, dev = _dtype(table, what), _device(table, what)
    bits = _ids(what, ids, dev)
    if table.dim() != 2:
        raise ValueError(f"{what}: table is [rows, width]")
    rows, width = table.shape
    ldt = _ld(what, "table", table, table.shape, table.dtype, dev)
    shape = (*ids.shape, width)
    if out is None:
        out, ldo = _new(shape, table.dtype, dev, stream), width
    else:
        ldo = _ld(what, "out", out, shape, table.dtype, dev)
    _call(LIB.kfac_embedding, "kfac_embedding", dev, stream,
          EMBEDDING_DESC.pack(dt, bits, ids.numel(), rows, width, float(scale), ldt, ldo),
          ids.data_ptr(), table.data_ptr(), out.data_ptr())
    return out


def embedding_workspace(ids, rows: int, width: int):
    """A workspace tensor for embedding_backward of as many ids or fewer, to be kept and passed to it."""
    dev = _device(ids, "embedding_workspace")
    return _kept(_sized(LIB.kfac_embedding_workspace_size, "kfac_embedding_workspace_size", dev,
                        ids.numel(), rows, width), dev)


def embedding_backward(ids, dout, rows: int, scale: float = 1.0, padding_id: int = -1, out=None,
                       accumulate: bool = False, frequency=None, workspace=None, stream=None):
    """kfac_embedding_backward: the gradient (float32 [rows, width]) of embedding's table for the
    gradient dout [..., width] of its out; returns out.  Tokens of padding_id (-1: none) and ids
    outside the table are left out.  accumulate=True adds to the given out, whose rows without
    tokens are not touched.  frequency (float32 [rows], given): each row's share of the tokens, which
    Kfac.diag_step takes as g_new of a layer of d_out = rows."""
    what = "embedding_backward"
    dt, dev = _dtype(dout, what), _device(dout, what)
    bits = _ids(what, ids, dev)
    if dout.dim() < 1 or dout.shape[:-1] != ids.shape:
        raise ValueError(f"{what}: dout is [..., width] for ids [...], not {tuple(dout.shape)}")
    if not -2**63 <= padding_id < 2**63:   # (ctypes would wrap it)
        raise ValueError(f"{what}: padding_id is an id, or -1 for none, not {padding_id}")
    width, tokens = dout.shape[-1], ids.numel()
    ldo = _ld(what, "dout", dout, dout.shape, dout.dtype, dev)
    if out is None:
        if accumulate:
            raise ValueError(f"{what}: accumulate adds to a given out")
        out = _new((rows, width), torch.float32, dev, stream)
    ldt = _ld(what, "out", out, (rows, width), torch.float32, dev)
    workspace = _workspace(what, workspace, 0 if workspace is not None else _sized(
        LIB.kfac_embedding_workspace_size, "kfac_embedding_workspace_size", dev, tokens, rows, width),
        dev, stream)
    _call(LIB.kfac_embedding_backward, "kfac_embedding_backward", dev, stream,
          EMBEDDING_DESC.pack(dt, bits, tokens, rows, width, float(scale), ldt, ldo),
          ids.data_ptr(), dout.data_ptr(), out.data_ptr(), padding_id, int(accumulate),
          _vector(what, "frequency", frequency, rows, dev), workspace.data_ptr(), workspace.nbytes)
    return out


# ----------------------------------------------------------------------- orthogonalised updates

_INT_MAX = 2**31 - 1


class _Matrices:
    """A list of 2-D tensors with contiguous rows (3-D ones: their entries) as the C call takes it."""

    def __init__(self, what, name, tensors, dtype=None, like=None):
        ts = []
        for t in ([tensors] if isinstance(tensors, torch.Tensor) else tensors):
            if t.dim() == 3:
                ts.extend(t.unbind(0))
            elif t.dim() == 2:
                ts.append(t)
            else:
                raise ValueError(f"{what}: {name} is [rows, columns], or [batch, rows, columns]")
        self.count = n = len(ts)
        if like is None:
            self.dev = _device(ts[0], what) if n else torch.cuda.current_device()
            self.dtype = ts[0].dtype if n else torch.float32
            self.dt = _dtype(ts[0], what) if n else 0
            self.shapes = [t.shape for t in ts]
            # (a side that no int holds is refused by the library, not wrapped)
            self.rows = (ctypes.c_int * n)(*[min(s[0], _INT_MAX) for s in self.shapes])
            self.cols = (ctypes.c_int * n)(*[min(s[1], _INT_MAX) for s in self.shapes])
        else:
            self.dev, self.dtype, self.shapes = like.dev, dtype or like.dtype, like.shapes
            if n != like.count:
                raise ValueError(f"{what}: {name} has {n} matrices, not {like.count}")
        lds = []
        for t, shape in zip(ts, self.shapes):
            if t.dtype is not self.dtype or t.shape != shape:
                raise ValueError(f"{what}: {name} holds {t.dtype} {tuple(t.shape)}, not {self.dtype} "
                                 f"{tuple(shape)}")
            if t.get_device() != self.dev:
                _elsewhere(what, name, t, self.dev)
            s0, s1 = t.stride()
            if s1 != 1 and shape[1] > 1:
                raise ValueError(f"{what}: {name}'s rows are contiguous")
            lds.append(s0)
        self.ld = (ctypes.c_int64 * n)(*lds)
        self.ptr = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ts])


def _ortho_desc(what, dt, math, steps, eps, coefficients):
    """(descriptor bytes, the coefficients that it points to)."""
    if math is None:
        math = KFAC_ORTHO_HALF if dt == KFAC_BF16 else KFAC_ORTHO_FULL
    flat = None
    if coefficients is not None:
        rows = list(coefficients)
        if len(rows) == 3 and not hasattr(rows[0], "__len__"):
            rows = [rows] * steps
        if len(rows) != steps or any(len(r) != 3 for r in rows):
            raise ValueError(f"{what}: coefficients are (a, b, c), or one such triple per step")
        flat = (ctypes.c_double * (3 * steps))(*[float(v) for r in rows for v in r])
    return ORTHO_DESC.pack(dt, math, steps, float(eps), ctypes.addressof(flat) if flat else 0), flat


def orthogonalize_workspace(x, math=None):
    """A workspace tensor for orthogonalize or orthogonal_step of matrices like x, or of some of them
    (tensor or list; orthogonal_step: the gradients), to be kept and passed to the calls."""
    what = "orthogonalize_workspace"
    m = _Matrices(what, "x", x)
    # (any number of steps but one takes the same)
    desc, _ = _ortho_desc(what, m.dt, math, 2, 0.0, None)
    return _kept(_sized(LIB.kfac_orthogonalize_workspace_size, "kfac_orthogonalize_workspace_size",
                        m.dev, desc, m.count, m.rows, m.cols), m.dev)


def _ortho_workspace(what, desc, m, workspace, stream):
    return _workspace(what, workspace, 0 if workspace is not None else _sized(
        LIB.kfac_orthogonalize_workspace_size, "kfac_orthogonalize_workspace_size", m.dev, desc,
        m.count, m.rows, m.cols), m.dev, stream)


def orthogonalize(x, out=None, steps: int = 5, coefficients=None, eps: float = 1e-7, math=None,
                  workspace=None, stream=None):
    """kfac_orthogonalize: the orthogonal factor of each matrix by Newton-Schulz products; returns
    out.  x: a tensor [rows, columns] or [batch, rows, columns], or a list of such, float32 or
    bfloat16, rows contiguous; out alike (may be x).  math: KFAC_ORTHO_FULL (the default for
    float32) or KFAC_ORTHO_HALF (for bfloat16).  coefficients: (a, b, c) of x -> a x + b x^3 + c x^5
    for every step, or one triple per step."""
    what = "orthogonalize"
    if not isinstance(x, torch.Tensor):
        x = list(x)   # (an iterator gives its tensors once)
    if out is not None and not isinstance(out, torch.Tensor):
        out = list(out)
    m = _Matrices(what, "x", x)
    if out is None:
        one = isinstance(x, torch.Tensor)
        new = [_new(t.shape, t.dtype, m.dev, stream) for t in ([x] if one else x)]
        out = new[0] if one else new
    o = _Matrices(what, "out", out, like=m)
    desc, keep = _ortho_desc(what, m.dt, math, steps, eps, coefficients)
    workspace = _ortho_workspace(what, desc, m, workspace, stream)
    _call(LIB.kfac_orthogonalize, "kfac_orthogonalize", m.dev, stream, desc, m.count, m.rows, m.cols,
          m.ptr, m.ld, o.ptr, o.ld, workspace.data_ptr(), workspace.nbytes)
    return out


def orthogonal_step(grads, momenta, params, lr: float, momentum: float = 0.95,
                    weight_decay: float = 0.0, nesterov: bool = True, update_scale: float = 1.0,
                    steps: int = 5, coefficients=None, eps: float = 1e-7, math=None, workspace=None,
                    stream=None):
    """kfac_orthogonal_step: one optimizer step of each matrix along its orthogonalised momentum.
    grads: as orthogonalize's x; momenta, params: float32 of the same shapes, updated in place.  math:
    as there, by the gradients' type: KFAC_ORTHO_HALF for bfloat16 ones, whatever the momenta are."""
    what = "orthogonal_step"
    g = _Matrices(what, "grads", grads)
    m = _Matrices(what, "momenta", momenta, torch.float32, like=g)
    p = _Matrices(what, "params", params, torch.float32, like=g)
    desc, keep = _ortho_desc(what, g.dt, math, steps, eps, coefficients)
    hp = ORTHO_STEP.pack(float(lr), float(momentum), float(weight_decay), float(update_scale),
                         bool(nesterov))
    workspace = _ortho_workspace(what, desc, g, workspace, stream)
    _call(LIB.kfac_orthogonal_step, "kfac_orthogonal_step", g.dev, stream, desc, hp, g.count, g.rows,
          g.cols, g.ptr, g.ld, m.ptr, m.ld, p.ptr, p.ld, workspace.data_ptr(), workspace.nbytes)
