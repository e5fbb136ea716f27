"""Operators between the linear layers of a transformer block: rotary positions, cross
attention to an encoder's states, dropout with the residual added; forward and backward.

Argument marshalling only, as in the rest of the package: outputs and workspace may be given
(a training loop keeps them) or are allocated with torch.  Activations are
[batch, length, heads, head_dim] tensors with contiguous channels and any other strides.  A
wrong shape, type or device raises ValueError; what the library itself refuses raises KfacError.
Definitions: include/kfac.h.

``stream``: a torch stream or a raw handle; torch's current stream of the tensors' device
unless one is given.  The inputs have to be ready there (as for every call of the package);
tensors allocated here are marked as used on it.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._lib import (LIB, KFAC_F32, KFAC_BF16, KFAC_ROPE_PLAIN, ROPE_DESC, ATTENTION_DESC,
                   ATTENTION_GRAD_DESC, KfacError)

_DTYPE = {torch.float32: KFAC_F32, torch.bfloat16: KFAC_BF16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_here = contextlib.nullcontext()


def _check(code: int, what: str):
    if code != 0:
        raise KfacError(code, what)


def _dtype(t, what):
    try:
        return _DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"{what}: float32 or bfloat16 tensors, not {t.dtype}") from None


def _same(what, ref, **tensors):
    """Every tensor on ref's CUDA device."""
    if not ref.is_cuda:
        raise ValueError(f"{what}: CUDA tensors (there is no CPU implementation)")
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{what}: {name} is on {t.device}, not {ref.device}")


def _heads(what, name, t, dtype, shape):
    """t: [batch, length, heads, head_dim] of this type and shape, channels contiguous."""
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{what}: {name} is {t.dtype} {tuple(t.shape)}, not {dtype} {tuple(shape)}")
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError(f"{what}: {name}'s channels are not contiguous (stride {s[3]})")
    return s


def _on(device):
    """The library works on the current device: make it the tensors'."""
    return _here if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _stream(stream, device):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _used_on(stream, device, *made):
    """Tensors allocated here belong to torch's current stream: tell its allocator where else
    they are used."""
    if stream is None:
        return
    s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
    for t in made:
        if t is not None:
            t.record_stream(s)


def _p(t):
    return None if t is None else t.data_ptr()


# --------------------------------------------------------------------------- rotary positions

def rope_table(rows: int, rotary_dim: int, base: float = 10000.0, scaling: int = KFAC_ROPE_PLAIN,
               factor: float = 1.0, original_length: float = 1.0, out=None, device=None,
               stream=None):
    """kfac_rope_table: the cosines and sines of positions 0..rows-1, float32
    [rows, rotary_dim].  scaling: KFAC_ROPE_PLAIN, KFAC_ROPE_LINEAR, KFAC_ROPE_NTK or
    KFAC_ROPE_YARN (which reads original_length), over a context ``factor`` times as long."""
    made = None
    if out is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        out = made = torch.empty(rows, rotary_dim, device=dev)
    _same("rope_table", out)
    if out.dtype != torch.float32 or out.shape != (rows, rotary_dim) or not out.is_contiguous():
        raise ValueError("rope_table: out is float32 [rows, rotary_dim], contiguous")
    with _on(out.device):
        _check(LIB.kfac_rope_table(out.data_ptr(), rows, rotary_dim, float(base), scaling,
                                   float(factor), float(original_length),
                                   _stream(stream, out.device)), "kfac_rope_table")
    _used_on(stream, out.device, made)
    return out


def rope(q, k, table, positions=None, position_offset: int = 0, interleaved: bool = False,
         inverse: bool = False, out_q=None, out_k=None, stream=None):
    """kfac_rope: rotary positions of q [batch, length, heads, head_dim] and k (either may be
    None) in one launch; returns (out_q, out_k).  The first table.shape[1] channels of each head
    turn.  positions: int32 [batch, length] or [length], or None for position_offset + row.
    inverse=True is the backward pass (gradients of the outputs in, of the inputs out).
    out_q=q, out_k=k work in place."""
    ref = q if q is not None else k
    if ref is None or ref.dim() != 4:
        raise ValueError("rope: q or k [batch, length, heads, head_dim]")
    _same("rope", ref, k=k, table=table, positions=positions, out_q=out_q, out_k=out_k)
    dt = _dtype(ref, "rope")
    b, n, _, d = ref.shape
    if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("rope: table is float32 [rows, rotary_dim], contiguous")
    made = [None, None]
    strides, heads = [], []
    for i, (name, x, y) in enumerate((("q", q, out_q), ("k", k, out_k))):
        if x is None:
            strides.append(((0, 0, 0, 0), (0, 0, 0, 0)))
            heads.append(0)
            continue
        h = x.shape[2] if x.dim() == 4 else 0
        shape = (b, n, h, d)
        sx = _heads("rope", name, x, ref.dtype, shape)
        if y is None:
            y = made[i] = torch.empty(shape, dtype=x.dtype, device=x.device)
            if i == 0:
                out_q = y
            else:
                out_k = y
        strides.append((sx, _heads("rope", "out_" + name, y, ref.dtype, shape)))
        heads.append(h)
    ps = 0
    if positions is not None:
        if positions.dtype != torch.int32 or positions.shape not in ((b, n), (n,)) or (
                n > 1 and positions.stride(-1) != 1):
            raise ValueError("rope: positions is int32 [batch, length] or [length], rows contiguous")
        ps = positions.stride(0) if positions.dim() == 2 else 0
    (qs, oq), (ks, ok) = strides
    desc = ROPE_DESC.pack(dt, b, n, heads[0], heads[1], d, table.shape[1], bool(interleaved),
                          bool(inverse), table.shape[0], position_offset, ps, qs[0], qs[1], qs[2],
                          ks[0], ks[1], ks[2], oq[0], oq[1], oq[2], ok[0], ok[1], ok[2])
    with _on(ref.device):
        _check(LIB.kfac_rope(desc, _p(q), _p(k), table.data_ptr(), _p(positions),
                             None if q is None else out_q.data_ptr(),
                             None if k is None else out_k.data_ptr(), _stream(stream, ref.device)),
               "kfac_rope")
    _used_on(stream, ref.device, *made)
    return (None if q is None else out_q), (None if k is None else out_k)


# ------------------------------------------------------------------------------------ dropout

def _rows(what, name, t, like):
    """(leading dimension) of a tensor read as [rows, cols] with contiguous columns."""
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{what}: {name} is {t.dtype} {tuple(t.shape)}, not {like.dtype} "
                         f"{tuple(like.shape)}")
    if t.dim() == 2 and (t.stride(1) == 1 or t.shape[1] <= 1):
        return t.stride(0)
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} is contiguous, or 2-D with contiguous rows")
    return t.shape[-1] if t.dim() else 1


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, out=None, stream=None):
    """kfac_dropout: residual + dropout(x) (residual may be None) with the mask of (seed, offset);
    returns out.  x: contiguous of any shape, or 2-D with contiguous rows.  Each use within a
    step takes an offset (or seed) of its own; the backward pass takes the same one."""
    dt = _dtype(x, "dropout")
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("dropout: seed and offset are 64-bit counts")
    _same("dropout", x, residual=residual, out=out)
    made = None
    if out is None:
        out = made = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    ldx, ldo = _rows("dropout", "x", x, x), _rows("dropout", "out", out, x)
    ldr = _rows("dropout", "residual", residual, x) if residual is not None else 0
    cols = x.shape[-1] if x.dim() else 1
    rows = x.numel() // cols if cols else 0
    with _on(x.device):
        _check(LIB.kfac_dropout(dt, x.data_ptr(), ldx, _p(residual), ldr, out.data_ptr(), ldo,
                                rows, cols, p, seed, offset, _stream(stream, x.device)),
               "kfac_dropout")
    _used_on(stream, x.device, made)
    return out


def dropout_backward(dout, p: float, seed: int, offset: int = 0, out=None, stream=None):
    """The gradient with respect to dropout's x, given that of its output (which is the gradient
    with respect to the residual): the same mask, generated again."""
    return dropout(dout, p, seed, offset, None, out, stream)


# ---------------------------------------------------------------------------- cross attention

def _attention(what, q, k, v, out, scale):
    """Descriptor bytes of these tensors."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError(f"{what}: q [batch, len_q, heads, head_dim], k [batch, len_kv, kv_heads, "
                         f"head_dim]")
    b, nq, h, d = q.shape
    nk, kv = k.shape[1], k.shape[2]
    qs = _heads(what, "q", q, q.dtype, q.shape)
    ks = _heads(what, "k", k, q.dtype, (b, nk, kv, d))
    vs = _heads(what, "v", v, q.dtype, (b, nk, kv, d)) if v is not None else ks
    os = _heads(what, "out", out, q.dtype, q.shape) if out is not None else qs
    return ATTENTION_DESC.pack(_dtype(q, what), b, nq, nk, h, kv, d,
                               0.0 if scale is None else scale, qs[0], qs[1], qs[2], ks[0], ks[1],
                               ks[2], vs[0], vs[1], vs[2], os[0], os[1], os[2])


def _keys(what, kv_len, key_mask, k):
    if kv_len is not None and (kv_len.dtype != torch.int32 or kv_len.shape != (k.shape[0],)
                               or not kv_len.is_contiguous()):
        raise ValueError(f"{what}: kv_len is int32 [batch], contiguous")
    if key_mask is not None and (key_mask.dtype not in (torch.uint8, torch.bool)
                                 or key_mask.shape != k.shape[:2] or not key_mask.is_contiguous()):
        raise ValueError(f"{what}: key_mask is uint8 or bool [batch, len_kv], contiguous")


def _workspace_bytes(desc, backward, device):
    nbytes = ctypes.c_size_t(0)
    with _on(device):
        _check(LIB.kfac_cross_attention_workspace_size(desc, int(backward), ctypes.byref(nbytes)),
               "kfac_cross_attention_workspace_size")
    return nbytes.value


def cross_attention_workspace(q, k, backward: bool = False):
    """A workspace tensor for cross_attention (backward=True: and cross_attention_backward) of
    tensors like these, to be kept and passed to the calls."""
    _same("cross_attention_workspace", q, k=k)
    desc = _attention("cross_attention_workspace", q, k, None, None, None)
    n = _workspace_bytes(desc, backward, q.device)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)


def cross_attention(q, k, v, kv_len=None, key_mask=None, scale=None, out=None, lse=None,
                    workspace=None, stream=None):
    """kfac_cross_attention: softmax(scale q k^T) v over the permitted keys; returns (out, lse).
    q [batch, len_q, heads, head_dim]; k, v [batch, len_kv, kv_heads, head_dim]; kv_len int32
    [batch] and key_mask uint8 or bool [batch, len_kv] say which keys are permitted (None: all);
    scale None: 1/sqrt(head_dim).  lse: float32 [batch, heads, len_q], kept for the backward
    pass."""
    _same("cross_attention", q, k=k, v=v, kv_len=kv_len, key_mask=key_mask, out=out, lse=lse,
          workspace=workspace)
    made = [None, None, None]
    if out is None:
        out = made[0] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    desc = _attention("cross_attention", q, k, v, out, scale)
    _keys("cross_attention", kv_len, key_mask, k)
    stats = (q.shape[0], q.shape[2], q.shape[1])
    if lse is None:
        lse = made[1] = torch.empty(stats, device=q.device)
    elif lse.dtype != torch.float32 or lse.shape != stats or not lse.is_contiguous():
        raise ValueError("cross_attention: lse is float32 [batch, heads, len_q], contiguous")
    if workspace is None:
        workspace = made[2] = torch.empty(_workspace_bytes(desc, False, q.device),
                                          dtype=torch.uint8, device=q.device)
    with _on(q.device):
        _check(LIB.kfac_cross_attention(desc, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        _p(kv_len), _p(key_mask), out.data_ptr(), lse.data_ptr(),
                                        workspace.data_ptr(),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream, q.device)), "kfac_cross_attention")
    _used_on(stream, q.device, *made)
    return out, lse


def cross_attention_backward(dout, q, k, v, out, lse, kv_len=None, key_mask=None, scale=None,
                             dq=None, dk=None, dv=None, workspace=None, stream=None):
    """kfac_cross_attention_backward: the gradients (dq, dk, dv) of cross_attention for the
    gradient dout of its output, from its inputs and its out and lse; dk and dv of a key head
    sum over the query heads that share it."""
    what = "cross_attention_backward"
    _same(what, q, dout=dout, k=k, v=v, out=out, lse=lse, kv_len=kv_len, key_mask=key_mask,
          dq=dq, dk=dk, dv=dv, workspace=workspace)
    desc = _attention(what, q, k, v, out, scale)
    _keys(what, kv_len, key_mask, k)
    if lse.dtype != torch.float32 or lse.shape != (q.shape[0], q.shape[2], q.shape[1]) or (
            not lse.is_contiguous()):
        raise ValueError(f"{what}: lse is float32 [batch, heads, len_q], contiguous")
    made = [None] * 4
    if dq is None:
        dq = made[0] = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if dk is None:
        dk = made[1] = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    if dv is None:
        dv = made[2] = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    grads = ATTENTION_GRAD_DESC.pack(*_heads(what, "dout", dout, q.dtype, q.shape)[:3],
                                     *_heads(what, "dq", dq, q.dtype, q.shape)[:3],
                                     *_heads(what, "dk", dk, q.dtype, k.shape)[:3],
                                     *_heads(what, "dv", dv, q.dtype, k.shape)[:3])
    if workspace is None:
        workspace = made[3] = torch.empty(_workspace_bytes(desc, True, q.device),
                                          dtype=torch.uint8, device=q.device)
    with _on(q.device):
        _check(LIB.kfac_cross_attention_backward(
            desc, grads, dout.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            out.data_ptr(), lse.data_ptr(), _p(kv_len), _p(key_mask), dq.data_ptr(),
            dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream(stream, q.device)),
            "kfac_cross_attention_backward")
    _used_on(stream, q.device, *made)
    return dq, dk, dv


def operator_status():
    """kfac_operator_status: synchronises; (code, info) of the first device error of these
    operators since the last call (code 0: none)."""
    info = ctypes.c_int(0)
    return LIB.kfac_operator_status(ctypes.byref(info)), info.value
