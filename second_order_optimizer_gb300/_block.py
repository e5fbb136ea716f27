"""Operators between the linear layers of a transformer block: rotary positions, cross
attention to an encoder's states, dropout with the residual added; forward and backward.

Argument marshalling only, as in the rest of the package: outputs and workspace may be given
(a training loop keeps them) or are allocated with torch.  Activations are
[batch, length, heads, head_dim] tensors with contiguous channels and any other strides.  A
wrong shape, type or device raises ValueError; what the library itself refuses raises KfacError.
The calls are outside torch's autograd, like the rest of the package: a result has no graph,
whatever its inputs require, and the backward passes here are called by hand.
Definitions: include/kfac.h.

``stream``: a torch stream or a raw handle; torch's current stream of the tensors' device
unless one is given.  The inputs have to be ready there (as for every call of the package);
tensors allocated here belong to it and are marked as used on the current one, where the
caller has to wait for it before reading them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._lib import (LIB, KFAC_F32, KFAC_BF16, KFAC_ROPE_PLAIN, ROPE_DESC, ATTENTION_DESC,
                   ATTENTION_GRAD_DESC, KfacError)

_DTYPE = {torch.float32: KFAC_F32, torch.bfloat16: KFAC_BF16}
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_MAX64 = (1 << 64) - 1
_F32_MIN, _F32_MAX = 2.0 ** -126, (2 - 2.0 ** -23) * 2.0 ** 127

# The checks below are spelled out call by call rather than looped over: a call of a few rows
# takes the GPU two microseconds, and each attribute of a tensor costs about 0.1.


def _check(code: int, what: str):
    if code != 0:
        raise KfacError(code, what)


def _dtype(t, what):
    dt = _DTYPE.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: float32 or bfloat16 tensors, not {t.dtype}")
    return dt


def _device(t, what):
    """The index of t's CUDA device."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{what}: CUDA tensors (there is no CPU implementation)")
    return dev


def _elsewhere(what, name, t, dev):
    raise ValueError(f"{what}: {name} is on {t.device}, not cuda:{dev}")


def _heads(what, name, t, dtype, shape, dev):
    """Strides of t: [batch, length, heads, head_dim] of this type, shape and device, channels
    contiguous."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what}: {name} is {t.dtype} {tuple(t.shape)}, not {dtype} {tuple(shape)}")
    if t.get_device() != dev:
        _elsewhere(what, name, t, dev)
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{what}: {name}'s channels are not contiguous (stride {s[3]})")
    return s


def _call(f, what, dev, stream, *args):
    """f(*args, stream) on the tensors' device (the library works on the current one)."""
    s = _raw_stream(dev) if stream is None else (
        stream if isinstance(stream, int) else stream.cuda_stream)
    if dev == _current_device():
        code = f(*args, s)
    else:
        with torch.cuda.device(dev):
            code = f(*args, s)
    if code != 0:
        raise KfacError(code, what)


def _empty(shape, dtype, dev, stream):
    """A tensor that ``stream`` (not None) may write at once.  torch hands out memory whose last
    use is still queued on the stream that it belongs to, which orders nothing on another: so it
    has to be that stream's own."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev)
    current, device = torch.cuda.current_stream(dev), torch.device("cuda", dev)
    if dev != _current_device():
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
    else:   # the same; the context takes 9 us more
        torch.cuda.set_stream(stream)
        try:
            t = torch.empty(shape, dtype=dtype, device=device)
        finally:
            torch.cuda.set_stream(current)
    t.record_stream(current)
    return t


# --------------------------------------------------------------------------- rotary positions

def rope_table(rows: int, rotary_dim: int, base: float = 10000.0, scaling: int = KFAC_ROPE_PLAIN,
               factor: float = 1.0, original_length: float = 1.0, out=None, device=None,
               stream=None):
    """kfac_rope_table: the cosines and sines of positions 0..rows-1, float32
    [rows, rotary_dim].  scaling: KFAC_ROPE_PLAIN, KFAC_ROPE_LINEAR, KFAC_ROPE_NTK or
    KFAC_ROPE_YARN (which reads original_length), over a context ``factor`` times as long."""
    if out is None:
        dev = None if device is None else torch.device(device)
        dev = torch.cuda.current_device() if dev is None or dev.index is None else dev.index
        if stream is None:
            out = torch.empty(rows, rotary_dim, device=torch.device("cuda", dev))
        else:
            out = _empty((rows, rotary_dim), torch.float32, dev, stream)
    dev = _device(out, "rope_table")
    if out.dtype != torch.float32 or out.shape != (rows, rotary_dim) or not out.is_contiguous():
        raise ValueError("rope_table: out is float32 [rows, rotary_dim], contiguous")
    _call(LIB.kfac_rope_table, "kfac_rope_table", dev, stream, out.data_ptr(), rows, rotary_dim,
          float(base), scaling, float(factor), float(original_length))
    return out


def rope(q, k, table, positions=None, position_offset: int = 0, interleaved: bool = False,
         inverse: bool = False, out_q=None, out_k=None, stream=None):
    """kfac_rope: rotary positions of q [batch, length, heads, head_dim] and k (either may be
    None) in one launch; returns (out_q, out_k).  The first table.shape[1] channels of each head
    turn.  positions: int32 [batch, length] or [length], or None for position_offset + row.
    inverse=True is the backward pass (gradients of the outputs in, of the inputs out).
    out_q=q, out_k=k work in place."""
    ref = q if q is not None else k
    if ref is None or ref.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("rope: q and k are [batch, length, heads, head_dim]")
    dt, dtype, dev = _dtype(ref, "rope"), ref.dtype, _device(ref, "rope")
    b, n, _, d = ref.shape
    if table.dtype is not torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("rope: table is float32 [rows, rotary_dim], contiguous")
    if table.get_device() != dev:
        _elsewhere("rope", "table", table, dev)
    h = kv = 0
    qs = ks = oqs = oks = (0, 0, 0, 0)
    if q is not None:
        shape, qs = q.shape, q.stride()
        h = shape[2]
        if out_q is None:
            out_q = (torch.empty(shape, dtype=dtype, device=q.device) if stream is None
                     else _empty(shape, dtype, dev, stream))
        oqs = out_q.stride()
        if out_q.shape != shape or out_q.dtype is not dtype or out_q.get_device() != dev or (
                d > 1 and (qs[3] != 1 or oqs[3] != 1)):
            _heads("rope", "q", q, dtype, shape, dev)
            _heads("rope", "out_q", out_q, dtype, shape, dev)
    if k is not None:
        shape, ks = k.shape, k.stride()
        kb, kn, kv, kd = shape
        if out_k is None:
            out_k = (torch.empty(shape, dtype=dtype, device=k.device) if stream is None
                     else _empty(shape, dtype, dev, stream))
        oks = out_k.stride()
        if kb != b or kn != n or kd != d or k.dtype is not dtype or k.get_device() != dev or (
                out_k.shape != shape or out_k.dtype is not dtype or out_k.get_device() != dev) or (
                d > 1 and (ks[3] != 1 or oks[3] != 1)):
            _heads("rope", "k", k, dtype, (b, n, kv, d), dev)
            _heads("rope", "out_k", out_k, dtype, (b, n, kv, d), dev)
    ps, pp = 0, None
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.shape not in ((b, n), (n,)) or (
                n > 1 and positions.stride(-1) != 1):
            raise ValueError("rope: positions is int32 [batch, length] or [length], rows contiguous")
        if positions.get_device() != dev:
            _elsewhere("rope", "positions", positions, dev)
        ps, pp = positions.stride(0) if positions.dim() == 2 else 0, positions.data_ptr()
    rows, rotary = table.shape
    desc = ROPE_DESC.pack(dt, b, n, h, kv, d, rotary, bool(interleaved), bool(inverse), rows,
                          position_offset, ps, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], oqs[0],
                          oqs[1], oqs[2], oks[0], oks[1], oks[2])
    _call(LIB.kfac_rope, "kfac_rope", dev, stream, desc, None if q is None else q.data_ptr(),
          None if k is None else k.data_ptr(), table.data_ptr(), pp,
          None if q is None else out_q.data_ptr(), None if k is None else out_k.data_ptr())
    return (None if q is None else out_q), (None if k is None else out_k)


# ------------------------------------------------------------------------------------ dropout

def _ld(name, t):
    """Leading dimension of a 2-D tensor with contiguous rows."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"dropout: {name} is contiguous, or 2-D with contiguous rows")
    return t.stride(0)


def _like(name, t, x, shape, dev):
    if t.shape != shape or t.dtype is not x.dtype:
        raise ValueError(f"dropout: {name} is {t.dtype} {tuple(t.shape)}, not {x.dtype} {tuple(shape)}")
    if t.get_device() != dev:
        _elsewhere("dropout", name, t, dev)


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, out=None, stream=None):
    """kfac_dropout: residual + dropout(x) (residual may be None) with the mask of (seed, offset);
    returns out.  x: contiguous of any shape, or 2-D with contiguous rows.  Each use within a
    step takes an offset (or seed) of its own; the backward pass takes the same one."""
    if not (0 <= seed <= _MAX64 and 0 <= offset <= _MAX64):
        raise ValueError("dropout: seed and offset are 64-bit counts")
    dt, shape, dev = _dtype(x, "dropout"), x.shape, _device(x, "dropout")
    rp = None
    if out is None:
        out = (torch.empty(shape, dtype=x.dtype, device=x.device) if stream is None
               else _empty(shape, x.dtype, dev, stream))
    else:
        _like("out", out, x, shape, dev)
    flat = x.is_contiguous() and out.is_contiguous()
    if residual is not None:
        _like("residual", residual, x, shape, dev)
        rp, flat = residual.data_ptr(), flat and residual.is_contiguous()
    if flat:   # the row-major index is the address
        rows, cols = 1, x.numel()
        ldx = ldr = ldo = cols
    else:
        ldx, ldo = _ld("x", x), _ld("out", out)
        ldr = _ld("residual", residual) if residual is not None else 0
        rows, cols = shape
    _call(LIB.kfac_dropout, "kfac_dropout", dev, stream, dt, x.data_ptr(), ldx, rp, ldr,
          out.data_ptr(), ldo, rows, cols, p, seed, offset)
    return out


def dropout_backward(dout, p: float, seed: int, offset: int = 0, out=None, stream=None):
    """The gradient with respect to dropout's x, given that of its output (which is the gradient
    with respect to the residual): the same mask, generated again."""
    return dropout(dout, p, seed, offset, None, out, stream)


# ---------------------------------------------------------------------------- cross attention

def _attention(what, q, k, v, out, scale, dev):
    """Descriptor bytes of these tensors (v and out None: laid out as k and q)."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"{what}: q [batch, len_q, heads, head_dim], k [batch, len_kv, kv_heads, "
                         f"head_dim]")
    dtype, shape, keys = q.dtype, q.shape, k.shape
    b, nq, h, d = shape
    kb, nk, kv, kd = keys
    qs, ks = q.stride(), k.stride()
    if kb != b or kd != d or k.dtype is not dtype or k.get_device() != dev or (
            d > 1 and (ks[3] != 1 or qs[3] != 1)):
        _heads(what, "q", q, dtype, shape, dev)
        _heads(what, "k", k, dtype, (b, nk, kv, d), dev)
    vs = _heads(what, "v", v, dtype, keys, dev) if v is not None else ks
    os = _heads(what, "out", out, dtype, shape, dev) if out is not None else qs
    if scale is None:
        scale = 0.0   # the library's default
    elif abs(scale) < _F32_MIN or _F32_MAX < abs(scale) < math.inf:   # (it refuses the other bad ones)
        raise ValueError(f"{what}: scale is a normal float32 number, not {scale} (None: 1/sqrt(head_dim))")
    return ATTENTION_DESC.pack(_dtype(q, what), b, nq, nk, h, kv, d, scale, qs[0], qs[1], qs[2], ks[0], ks[1],
                               ks[2], vs[0], vs[1], vs[2], os[0], os[1], os[2])


def _keys(what, kv_len, key_mask, k, dev):
    """Addresses of kv_len and key_mask, checked."""
    lp = mp = None
    if kv_len is not None:
        if kv_len.dtype is not torch.int32 or kv_len.shape != k.shape[:1] or (
                not kv_len.is_contiguous()):
            raise ValueError(f"{what}: kv_len is int32 [batch], contiguous")
        if kv_len.get_device() != dev:
            _elsewhere(what, "kv_len", kv_len, dev)
        lp = kv_len.data_ptr()
    if key_mask is not None:
        if key_mask.dtype not in (torch.uint8, torch.bool) or key_mask.shape != k.shape[:2] or (
                not key_mask.is_contiguous()):
            raise ValueError(f"{what}: key_mask is uint8 or bool [batch, len_kv], contiguous")
        if key_mask.get_device() != dev:
            _elsewhere(what, "key_mask", key_mask, dev)
        mp = key_mask.data_ptr()
    return lp, mp


def _stats(what, lse, q, dev):
    if lse.dtype is not torch.float32 or lse.shape != (q.shape[0], q.shape[2], q.shape[1]) or (
            not lse.is_contiguous()):
        raise ValueError(f"{what}: lse is float32 [batch, heads, len_q], contiguous")
    if lse.get_device() != dev:
        _elsewhere(what, "lse", lse, dev)


def _workspace_bytes(desc, backward, dev):
    nbytes = ctypes.c_size_t(0)
    with torch.cuda.device(dev):   # the plan depends on the device's SM count
        _check(LIB.kfac_cross_attention_workspace_size(desc, int(backward), ctypes.byref(nbytes)),
               "kfac_cross_attention_workspace_size")
    return nbytes.value


def _workspace(desc, backward, dev, stream):
    """A call's own workspace."""
    n = _workspace_bytes(desc, backward, dev)
    return (torch.empty(n, dtype=torch.uint8, device=torch.device("cuda", dev)) if stream is None
            else _empty((n,), torch.uint8, dev, stream))


def cross_attention_workspace(q, k, backward: bool = False):
    """A workspace tensor for cross_attention (backward=True: and cross_attention_backward) of
    tensors like these, to be kept and passed to the calls."""
    what = "cross_attention_workspace"
    dev = _device(q, what)
    n = _workspace_bytes(_attention(what, q, k, None, None, None, dev), backward, dev)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def cross_attention(q, k, v, kv_len=None, key_mask=None, scale=None, out=None, lse=None,
                    workspace=None, stream=None):
    """kfac_cross_attention: softmax(scale q k^T) v over the permitted keys; returns (out, lse).
    q [batch, len_q, heads, head_dim]; k, v [batch, len_kv, kv_heads, head_dim]; kv_len int32
    [batch] and key_mask uint8 or bool [batch, len_kv] say which keys are permitted (None: all);
    scale (above 0) None: 1/sqrt(head_dim).  lse: float32 [batch, heads, len_q], kept for the backward
    pass."""
    what = "cross_attention"
    dev = _device(q, what)
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device) if stream is None
               else _empty(q.shape, q.dtype, dev, stream))
    desc = _attention(what, q, k, v, out, scale, dev)
    lp, mp = _keys(what, kv_len, key_mask, k, dev)
    if lse is None:
        rows = (q.shape[0], q.shape[2], q.shape[1])
        lse = (torch.empty(rows, device=q.device) if stream is None
               else _empty(rows, torch.float32, dev, stream))
    else:
        _stats(what, lse, q, dev)
    if workspace is None:
        workspace = _workspace(desc, False, dev, stream)
    elif workspace.get_device() != dev:
        _elsewhere(what, "workspace", workspace, dev)
    _call(LIB.kfac_cross_attention, "kfac_cross_attention", dev, stream, desc, q.data_ptr(),
          k.data_ptr(), v.data_ptr(), lp, mp, out.data_ptr(), lse.data_ptr(),
          workspace.data_ptr(), workspace.nbytes)
    return out, lse


def cross_attention_backward(dout, q, k, v, out, lse, kv_len=None, key_mask=None, scale=None,
                             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """kfac_cross_attention_backward: the gradients (dq, dk, dv) of cross_attention for the
    gradient dout of its output, from its inputs and its out and lse; dk and dv of a key head
    sum over the query heads that share it."""
    what = "cross_attention_backward"
    dev = _device(q, what)
    desc = _attention(what, q, k, v, out, scale, dev)
    lp, mp = _keys(what, kv_len, key_mask, k, dev)
    _stats(what, lse, q, dev)
    dtype, shape, keys = q.dtype, q.shape, k.shape
    if dq is None:
        dq = (torch.empty(shape, dtype=dtype, device=q.device) if stream is None
              else _empty(shape, dtype, dev, stream))
    if dk is None:
        dk = (torch.empty(keys, dtype=dtype, device=q.device) if stream is None
              else _empty(keys, dtype, dev, stream))
    if dv is None:
        dv = (torch.empty(keys, dtype=dtype, device=q.device) if stream is None
              else _empty(keys, dtype, dev, stream))
    gs = _heads(what, "dout", dout, dtype, shape, dev)
    qs = _heads(what, "dq", dq, dtype, shape, dev)
    ks = _heads(what, "dk", dk, dtype, keys, dev)
    vs = _heads(what, "dv", dv, dtype, keys, dev)
    grads = ATTENTION_GRAD_DESC.pack(gs[0], gs[1], gs[2], qs[0], qs[1], qs[2], ks[0], ks[1], ks[2],
                                     vs[0], vs[1], vs[2])
    if workspace is None:
        workspace = _workspace(desc, True, dev, stream)
    elif workspace.get_device() != dev:
        _elsewhere(what, "workspace", workspace, dev)
    _call(LIB.kfac_cross_attention_backward, "kfac_cross_attention_backward", dev, stream, desc,
          grads, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
          lse.data_ptr(), lp, mp, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
          workspace.data_ptr(), workspace.nbytes)
    return dq, dk, dv


def operator_status():
    """kfac_operator_status: synchronises the current device; (code, info) of the first device
    error of these operators on it since the last call (code 0: none)."""
    info = ctypes.c_int(0)
    return LIB.kfac_operator_status(ctypes.byref(info)), info.value
