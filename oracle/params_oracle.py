"""Float64 reference of the operators of the parameters without Kronecker factors: root-mean-square
norms, the token embedding, orthogonalised updates.  NumPy, plain and slow; shares no code with the
GPU path."""
from __future__ import annotations

import numpy as np


def rms_norm(x, gain=None, residual=None, eps=1e-6):
    """(y, s, r): s = x + residual, r = (mean s^2 + eps)^(-1/2) per row, y = s r gain."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    r = 1.0 / np.sqrt((s * s).mean(axis=-1) + eps)
    y = s * r[..., None] * (1.0 if gain is None else np.asarray(gain, np.float64))
    return y, s, r


def rms_norm_backward(dy, h, gain, r, dh=None):
    """(dx, dgain, dgain_square) from the forward pass's h and r."""
    h, dy = np.asarray(h, np.float64), np.asarray(dy, np.float64)
    n = h * r[..., None]
    w = dy * (1.0 if gain is None else np.asarray(gain, np.float64))
    dx = r[..., None] * (w - n * (w * n).mean(axis=-1, keepdims=True))
    each = (dy * n).reshape(-1, h.shape[-1])
    return (dx if dh is None else dx + dh), each.sum(axis=0), (each * each).mean(axis=0)


def e4m3(v):
    """v rounded to 8 bits: three mantissa bits (ties to even), least exponent -6, largest value 448."""
    v = np.asarray(v, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -40)))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantize(y, group=0):
    """(q, scales): the largest magnitude of each group of channels (0: of the row) becomes 448."""
    cols = y.shape[-1]
    group = group or cols
    q, scales = np.zeros_like(y), []
    for c in range(0, cols, group):
        top = np.abs(y[..., c:c + group]).max(axis=-1) / 448.0
        scales.append(top)
        q[..., c:c + group] = e4m3(y[..., c:c + group] / np.where(top > 0, top, 1.0)[..., None])
    return q, np.stack(scales, axis=-1)


def embedding(ids, table, scale=1.0):
    ids, table = np.asarray(ids), np.asarray(table, np.float64)
    out = np.full((*ids.shape, table.shape[1]), np.nan)
    ok = (ids >= 0) & (ids < table.shape[0])
    out[ok] = scale * table[ids[ok]]
    return out


def embedding_backward(ids, dout, rows, scale=1.0, padding_id=-1):
    """(dtable, frequency): a sum over the tokens of each row, one token at a time."""
    ids = np.asarray(ids).reshape(-1)
    dout = np.asarray(dout, np.float64).reshape(ids.size, -1)
    dtable, count = np.zeros((rows, dout.shape[1])), np.zeros(rows)
    for t, v in enumerate(ids):
        if 0 <= v < rows and v != padding_id:
            dtable[v] += scale * dout[t]
            count[v] += 1
    return dtable, count / max(1, ids.size)


COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """Singular values mapped by the steps' polynomials, the singular vectors kept."""
    x = np.asarray(x, np.float64)
    norm = np.sqrt((x * x).sum()) + eps
    if norm == 0:
        return x.copy()
    u, t, vt = np.linalg.svd(x / norm, full_matrices=False)
    per_step = [coefficients] * steps if np.ndim(coefficients) == 1 else coefficients
    for a, b, c in per_step:
        t = a * t + b * t ** 3 + c * t ** 5
    return (u * t) @ vt


def newton_schulz(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """The same by its products."""
    x = np.asarray(x, np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    a, b, c = coefficients
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * g @ g) @ x
    return x


def orthogonal_step(grad, m, w, lr, momentum=0.95, weight_decay=0.0, nesterov=True, update_scale=1.0,
                    **kw):
    """(momentum, weights) after one step."""
    m = momentum * np.asarray(m, np.float64) + grad
    o = orthogonalize(grad + momentum * m if nesterov else m, **kw)
    scale = update_scale * np.sqrt(max(1.0, w.shape[0] / w.shape[1]))
    return m, w - lr * (scale * o + weight_decay * w)


def newton_schulz_fp16(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7, groups=None, mirror=False):
    """The products with every matrix between them rounded to fp16's 11 bits (x too): the error that
    such operands cannot avoid.  groups: sizes of the groups of steps taken on the small side before x
    is formed (None: single steps).  mirror: of the products on the small side the upper half is stored
    on both sides, so that their roundings are equal in pairs."""
    def near(v):
        m, e = np.frexp(v)
        return np.ldexp(np.rint(m * 2.0 ** 11), e - 11)

    def both(v):
        v = near(v)
        return np.triu(v) + np.triu(v, 1).T if mirror else v
    x = np.asarray(x, np.float64)
    x = x.T if x.shape[0] > x.shape[1] else x
    x = near(x) / (np.sqrt((x * x).sum()) + eps)
    a, b, c = coefficients
    eye = np.eye(x.shape[0])
    k = 0
    for size in groups or [1] * steps:
        g, p = near(x @ x.T), None
        for j in range(size):
            m = near(a * eye + b * g + c * g @ g)
            p = m if p is None else both(m @ p)
            if j + 1 < size:
                g = both(both(g @ m) @ m)
        k += size
        x = p @ x
        x = x if k == steps else near(x)
    return x
