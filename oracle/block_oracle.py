"""Float64 reference of the operators between a transformer block's linear layers: rotary
positions, cross attention with its gradients, dropout from a counter-based generator.  NumPy,
plain and slow; shares no code with the GPU path."""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rotary_dim, base=10000.0, scaling="plain", factor=1.0, original_length=1.0):
    """(frequencies [rotary_dim/2], magnitude) of a rotary table."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    f = float(base) ** (-2.0 * i / rotary_dim)
    if scaling == "plain":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        b = base * factor ** (rotary_dim / (rotary_dim - 2.0))
        return b ** (-2.0 * i / rotary_dim), 1.0
    assert scaling == "yarn"

    def index_of(turns):   # the (real) pair index that turns this often in original_length
        return rotary_dim * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

    low = max(math.floor(index_of(32)), 0)
    high = min(math.ceil(index_of(1)), rotary_dim - 1)
    if high <= low:
        high = low + 0.001
    r = np.clip((i - low) / (high - low), 0.0, 1.0)
    return f * (1 - r) + f / factor * r, 0.1 * math.log(factor) + 1.0


def rope_table(rows, rotary_dim, **kw):
    f, mag = rope_frequencies(rotary_dim, **kw)
    angle = np.arange(rows, dtype=np.float64)[:, None] * f
    return np.concatenate([np.cos(angle), np.sin(angle)], axis=1) * mag


def rope(x, table, positions, interleaved=False, inverse=False):
    """x [batch, length, heads, dim], positions [batch, length] -> rotated copy."""
    r = table.shape[1]
    half = r // 2
    x = np.asarray(x, np.float64)
    y = x.copy()
    t = np.asarray(table, np.float64)[positions][:, :, None, :]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = t[..., i], t[..., half + i] * (-1.0 if inverse else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def philox4x32(counter, key, rounds=10):
    """Philox4x32 of Salmon et al. (SC 2011): counter 4 words, key 2 words (Python ints)."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(rounds):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & m, (a >> 32) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def dropout_words(n, seed, offset):
    """The n random words u_i of a dropout call."""
    key = (seed & 0xFFFFFFFF, seed >> 32)
    out = []
    for blk in range((n + 3) // 4):
        out += philox4x32((blk & 0xFFFFFFFF, blk >> 32, offset & 0xFFFFFFFF, offset >> 32), key)
    return np.array(out[:n], dtype=np.uint64)


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, np.float64)
    keep = (dropout_words(x.size, seed, offset) >= math.floor(p * 2.0 ** 32)).reshape(x.shape)
    y = np.zeros_like(x)
    if p < 1.0:
        y[keep] = x[keep] / (1.0 - p)
    return y if residual is None else y + np.asarray(residual, np.float64)


def permitted(batch, len_kv, kv_len=None, key_mask=None):
    ok = np.ones((batch, len_kv), bool)
    if kv_len is not None:
        ok &= np.arange(len_kv)[None, :] < np.asarray(kv_len)[:, None]
    if key_mask is not None:
        ok &= np.asarray(key_mask) != 0
    return ok


def cross_attention(q, k, v, ok, scale=None):
    """q [b, nq, h, d], k, v [b, nk, kv, d], ok [b, nk] -> out, lse [b, h, nq]."""
    b, nq, h, d = q.shape
    kv = k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((b, nq, h, d)), np.full((b, h, nq), -np.inf)
    for i in range(b):
        at = np.nonzero(ok[i])[0]
        if at.size == 0:
            continue
        for j in range(h):
            s = scale * (q[i, :, j].astype(np.float64) @ k[i, at, j * kv // h].astype(np.float64).T)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(axis=1, keepdims=True)
            out[i, :, j] = (p / total) @ v[i, at, j * kv // h].astype(np.float64)
            lse[i, j] = (m + np.log(total))[:, 0]
    return out, lse


def cross_attention_backward(dout, q, k, v, ok, scale=None):
    """Gradients (dq, dk, dv) of sum(dout * out)."""
    b, nq, h, d = q.shape
    nk, kv = k.shape[1], k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    dq, dk, dv = np.zeros((b, nq, h, d)), np.zeros((b, nk, kv, d)), np.zeros((b, nk, kv, d))
    for i in range(b):
        at = np.nonzero(ok[i])[0]
        if at.size == 0:
            continue
        for j in range(h):
            n = j * kv // h
            qq, kk, vv, g = (np.asarray(t, np.float64) for t in
                             (q[i, :, j], k[i, at, n], v[i, at, n], dout[i, :, j]))
            s = scale * qq @ kk.T
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            dp = g @ vv.T
            ds = p * (dp - (p * dp).sum(axis=1, keepdims=True))
            dq[i, :, j] = scale * ds @ kk
            dk[i, at, n] += scale * ds.T @ qq
            dv[i, at, n] += p.T @ g
    return dq, dk, dv


def gradient_norm_bounds(dout, q, k, v, ok, scale=None, from_products=128):
    """(gradients, bounds): dq, dk, dv in float64, and how far from them in norm the roundings of
    bf16 may take an implementation that rounds P, dS and the results once each and, for sequences
    of more than ``from_products`` permitted keys, takes delta from the rounded out.

    u = 2^-8; a rounding is off by at most u and by u / sqrt(3) in the root mean square, so 1.5 u of
    the gradient's norm holds three of them with room.  A row's delta is off by
    u / sqrt(3) |dout out|, and with it the row's whole dS by P times that: scale P k in dq, and in dk
    scale P q, where the rows' errors are independent.  Twice its root mean square is allowed."""
    b, nq, h, d = q.shape
    kv = k.shape[2]
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    u = 2.0 ** -8
    grads = cross_attention_backward(dout, q, k, v, ok, scale)
    off = [0.0, 0.0]
    for i in range(b):
        at = np.nonzero(ok[i])[0]
        if at.size <= from_products:
            continue
        for j in range(h):
            n = j * kv // h
            qq, kk, vv, g = (np.asarray(t, np.float64) for t in
                             (q[i, :, j], k[i, at, n], v[i, at, n], dout[i, :, j]))
            s = scale * qq @ kk.T
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            e = (u * scale) ** 2 / 3 * ((g * (p @ vv)) ** 2).sum(axis=1)
            off[0] += (e * ((p @ kk) ** 2).sum(axis=1)).sum()
            off[1] += (e * (qq ** 2).sum(axis=1) * (p ** 2).sum(axis=1)).sum()
    off.append(0.0)
    return grads, [1.5 * u * np.linalg.norm(x) + 2 * math.sqrt(o) for x, o in zip(grads, off)]
