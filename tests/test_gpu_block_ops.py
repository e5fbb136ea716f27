"""GPU parity of the block operators (rotary positions, dropout, cross attention and its
gradients) with the float64 reference.

Tolerances, fixed before the first run.  u = 2^-8 bounds a rounding to bf16, 2^-24 one to fp32.
 * rope, dropout: fp32 arithmetic (a few roundings of the terms) and one rounding of the result.
 * cross attention: element by element, from the magnitudes of the sums.  bf16 inputs: the
   probabilities and dS enter their products rounded once (u), the result is rounded once (u),
   and delta inherits the rounding of out; fp32 sums of n terms and fp32 scores of 128 terms add
   n 2^-24 and the like: SLACK = 2e-5 of the sum of magnitudes covers both (len <= 4096 sums are
   accumulated in tiles).  fp32 inputs: SLACK alone.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import second_order_optimizer_gb300 as K  # noqa: E402
from oracle import block_oracle as B  # noqa: E402

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SLACK = 2e-5
BF16, F32 = torch.bfloat16, torch.float32


def _randn(seed, *shape, dtype=F32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, tol):
    got = _np(got)
    assert got.shape == ref.shape
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) - tol
    assert (bad <= 0).all(), (np.unravel_index(bad.argmax(), bad.shape), bad.max())


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert K.operator_status() == (0, 0)


# --------------------------------------------------------------------------------------- rope

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("b,n,h,kv,d,r", [
    (2, 5, 4, 2, 64, 64), (1, 1, 1, 1, 2, 2), (3, 17, 3, 1, 80, 32), (2, 33, 5, 5, 36, 20),
    (1, 7, 9, 3, 33, 6), (2, 3, 8, 2, 128, 128), (1, 130, 2, 1, 96, 24), (2, 4, 6, 0, 40, 40)])
def test_rope(dtype, interleaved, b, n, h, kv, d, r):
    q = _randn(1, b, n, h, d, dtype=dtype)
    k = _randn(2, b, n, kv, d, dtype=dtype) if kv else None
    table = K.rope_table(300, r)
    rng = np.random.default_rng(3)
    for positions, inverse in ((None, False), (rng.integers(0, 300, (b, n)), True),
                               (rng.integers(0, 300, n), False)):
        pt = None if positions is None else torch.from_numpy(positions.astype(np.int32)).cuda()
        off = 11 if positions is None else 0
        oq, ok = K.rope(q, k, table, positions=pt, position_offset=off, interleaved=interleaved,
                        inverse=inverse)
        at = np.broadcast_to(np.arange(n) + off if positions is None else positions, (b, n))
        for x, y in ((q, oq), (k, ok)):
            if x is None:
                assert y is None
                continue
            ref = B.rope(_np(x), _np(table), at, interleaved, inverse)
            # two products and their sum in fp32, one rounding of the result
            mags = B.rope(np.abs(_np(x)), np.abs(_np(table)) + 1, at, interleaved)
            _close(y, ref, 4 * 2.0 ** -24 * (np.abs(mags) + np.abs(_np(x)).max()) + U[dtype] * np.abs(ref))
            assert torch.equal(y[..., r:], x[..., r:])


def test_rope_strides_and_in_place():
    """q and k as parts of one packed buffer, heads before rows, in place and out of place."""
    b, n, h, kv, d = 2, 19, 4, 2, 64
    packed = _randn(5, b, n, (h + 2 * kv) * d + 8, dtype=BF16)
    q = packed[..., :h * d].unflatten(-1, (h, d))
    k = packed[..., h * d:(h + kv) * d].unflatten(-1, (kv, d))
    rest = packed[..., (h + kv) * d:].clone()
    table = K.rope_table(64, d)
    oq = torch.empty(b, h, n, d, device="cuda", dtype=BF16).transpose(1, 2)
    oq, ok = K.rope(q, k, table, out_q=oq)
    want = K.rope(q.contiguous(), k.contiguous(), table)
    assert torch.equal(oq, want[0]) and torch.equal(ok, want[1])
    K.rope(q, k, table, out_q=q, out_k=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(packed[..., (h + kv) * d:], rest)


def test_rope_positions_outside_the_table_give_nan():
    q = _randn(1, 1, 4, 2, 8)
    table = K.rope_table(10, 4)
    pos = torch.tensor([[0, -1, 10, 9]], dtype=torch.int32, device="cuda")
    y, _ = K.rope(q, None, table, positions=pos)
    bad = torch.isnan(y[..., :4]).all(dim=-1).all(dim=-1)[0].tolist()
    assert bad == [False, True, True, False]
    assert torch.equal(y[..., 4:], q[..., 4:])
    with pytest.raises(K.KfacError):
        K.rope(q, None, table, position_offset=7)


@pytest.mark.parametrize("scaling,name", [(K.KFAC_ROPE_PLAIN, "plain"), (K.KFAC_ROPE_LINEAR, "linear"),
                                          (K.KFAC_ROPE_NTK, "ntk"), (K.KFAC_ROPE_YARN, "yarn")])
@pytest.mark.parametrize("r", [2, 20, 128])
def test_rope_table(scaling, name, r):
    if name == "ntk" and r == 2:
        pytest.skip("the base is stretched by factor^(R/(R-2))")
    kw = dict(base=10000.0, factor=8.0, original_length=4096)
    t = K.rope_table(33000, r, scaling=scaling, **kw)
    ref = B.rope_table(33000, r, scaling=name, **kw)
    # one rounding to fp32; the angle's relative error of a few 2^-53 times 33000 rad
    _close(t, ref, 2.0 ** -24 * np.abs(ref) + 33000 * 16 * 2.0 ** -53)


def test_rope_gradient_is_the_inverse():
    """<dy, rope(x)> = <rope_inverse(dy), x> for every x: the transpose."""
    x, dy = _randn(1, 2, 9, 3, 24), _randn(2, 2, 9, 3, 24)
    table = K.rope_table(16, 12, scaling=K.KFAC_ROPE_YARN, factor=4.0, original_length=64)
    y, _ = K.rope(x, None, table, interleaved=True)
    dx, _ = K.rope(dy, None, table, interleaved=True, inverse=True)
    a, c = float((dy.double() * y.double()).sum()), float((dx.double() * x.double()).sum())
    size = float((dy.double().abs() * y.double().abs()).sum())
    assert abs(a - c) <= 8 * 2.0 ** -24 * size


# ------------------------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 5), (17, 33), (64, 128), (5, 1027)])
@pytest.mark.parametrize("p", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(dtype, rows, cols, p, residual):
    x = _randn(1, rows, cols, dtype=dtype)
    r = _randn(2, rows, cols, dtype=dtype) if residual else None
    seed, offset = (1 << 63) + 12345, (1 << 40) + 9
    y = K.dropout(x, p, seed, offset, residual=r)
    ref = B.dropout(_np(x), p, seed, offset, None if r is None else _np(r))
    mag = np.abs(_np(x)) / max(1 - p, 1e-9) * (p < 1) + (np.abs(_np(r)) if residual else 0)
    _close(y, ref, 3 * 2.0 ** -24 * mag + U[dtype] * np.abs(ref))
    if not residual:   # the mask itself, to the bit
        assert np.array_equal(_np(y) != 0, (ref != 0))
        dx = K.dropout_backward(torch.ones_like(x), p, seed, offset)
        assert np.array_equal(_np(dx) != 0, B.dropout(np.ones((rows, cols)), p, seed, offset) != 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dropout_strides_alignment_and_aliasing(dtype):
    """Rows within a wider buffer, a base that is not 16-byte aligned, the result over x or the
    residual: the same values as the contiguous call."""
    rows, cols = 9, 37
    x, r = _randn(1, rows, cols, dtype=dtype), _randn(2, rows, cols, dtype=dtype)
    want = K.dropout(x, 0.3, 5, 6, residual=r)
    wide = torch.zeros(rows, cols + 11, device="cuda", dtype=dtype)
    xs = wide[:, 3:3 + cols]
    xs.copy_(x)
    out = torch.zeros(rows, 2 * cols, device="cuda", dtype=dtype)
    assert torch.equal(K.dropout(xs, 0.3, 5, 6, residual=r, out=out[:, :cols]), want)
    assert (out[:, cols:] == 0).all()
    odd = torch.zeros(rows * cols + 1, device="cuda", dtype=dtype)[1:].view(rows, cols)
    odd.copy_(x)
    assert torch.equal(K.dropout(odd, 0.3, 5, 6, residual=r), want)
    y = r.clone()
    assert torch.equal(K.dropout(x, 0.3, 5, 6, residual=y, out=y), want)
    y = x.clone()
    assert torch.equal(K.dropout(y, 0.3, 5, 6, residual=r, out=y), want)
    assert torch.equal(K.dropout(x.view(3, 3, cols), 0.3, 5, 6, residual=r.view(3, 3, cols)).view(rows, cols), want)


def test_dropout_does_not_spread_what_it_drops():
    x = torch.full((64, 64), float("inf"), device="cuda")
    x[::2] = float("nan")
    keep = _np(K.dropout(torch.ones_like(x), 0.5, 1, 2)) != 0
    y = _np(K.dropout(x, 0.5, 1, 2, residual=torch.ones_like(x)))
    assert (y[~keep] == 1).all() and not np.isfinite(y[keep]).any()


# ---------------------------------------------------------------------------- cross attention

def _inputs(dtype, b, nq, nk, h, kv, d, keys, seed=0):
    q, k, v, g = (_randn(seed + i, *s, dtype=dtype) for i, s in enumerate(
        [(b, nq, h, d), (b, nk, kv, d), (b, nk, kv, d), (b, nq, h, d)]))
    kv_len = mask = None
    rng = np.random.default_rng(seed)
    if keys in ("len", "both"):
        kv_len = rng.integers(0, nk + 1, b).astype(np.int32)
        kv_len[0] = 0 if b > 1 else max(nk - 1, 0)
    if keys in ("mask", "both"):
        mask = (rng.random((b, nk)) < 0.6).astype(np.uint8)
        if b > 1:
            mask[-1] = 0
    ok = B.permitted(b, nk, kv_len, mask)
    bad = torch.from_numpy(~ok).cuda()
    k[bad], v[bad] = float("nan"), float("inf")
    to = lambda x: None if x is None else torch.from_numpy(x).cuda()
    return q, k, v, g, to(kv_len), to(mask), ok


def _bounds(q, k, v, g, ok, scale, dtype):
    """Reference values and the magnitudes of their sums (float64 arrays)."""
    b, nq, h, d = q.shape
    kv = k.shape[2]
    u = U[dtype] if dtype == BF16 else 0.0   # rounding of P and dS as operands
    uo = U[dtype]
    z = lambda t: np.zeros(t.shape)
    r = {n: [z(t), z(t)] for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", v))}
    lse = np.full((b, h, nq), -np.inf)
    lse_tol = np.zeros((b, h, nq))
    for i in range(b):
        at = np.nonzero(ok[i])[0]
        if at.size == 0:
            continue
        for j in range(h):
            n = j * kv // h
            Q, Kk, V, G = q[i, :, j], k[i, at, n], v[i, at, n], g[i, :, j]
            s = scale * Q @ Kk.T
            ds_abs = scale * np.abs(Q) @ np.abs(Kk).T      # magnitude of each score's sum
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            lse[i, j] = (top + np.log(p.sum(axis=1, keepdims=True)))[:, 0]
            lse_tol[i, j] = 4e-6 * (1 + ds_abs.max(axis=1) + np.abs(lse[i, j]))
            p /= p.sum(axis=1, keepdims=True)
            pe = p * (u + SLACK * (1 + ds_abs))             # error of P
            o = p @ V
            oe = pe @ np.abs(V) + p @ np.abs(V) * SLACK
            dp = G @ V.T
            delta = (p * dp).sum(axis=1, keepdims=True)
            delta_e = (np.abs(G) * (oe + uo * np.abs(o))).sum(axis=1, keepdims=True) + SLACK * (
                np.abs(G) * np.abs(o)).sum(axis=1, keepdims=True)
            ds = p * (dp - delta)
            dse = (u * np.abs(ds) + p * SLACK * (1 + ds_abs) * np.abs(dp - delta)
                   + p * (SLACK * np.abs(G) @ np.abs(V).T + delta_e))
            for name, val, err, where in (
                    ("out", o, oe, (i, slice(None), j)),
                    ("dq", scale * ds @ Kk, scale * (dse + SLACK * np.abs(ds)) @ np.abs(Kk), (i, slice(None), j)),
                    ("dk", scale * ds.T @ Q, scale * (dse + SLACK * np.abs(ds)).T @ np.abs(Q), (i, at, n)),
                    ("dv", p.T @ G, (pe + SLACK * p).T @ np.abs(G), (i, at, n))):
                r[name][0][where] += val
                r[name][1][where] += err
    for name in r:
        r[name][1] += uo * (np.abs(r[name][0]) + r[name][1]) + 1e-30
    return r, lse, lse_tol


def _check_attention(q, k, v, g, kv_len, mask, ok, scale=None, stream=None, backward=True):
    dtype, d = q.dtype, q.shape[3]
    out, lse = K.cross_attention(q, k, v, kv_len, mask, scale=scale, stream=stream)
    grads = (K.cross_attention_backward(g, q, k, v, out, lse, kv_len, mask, scale=scale,
                                        stream=stream) if backward else None)
    torch.cuda.synchronize()
    r, lse_ref, lse_tol = _bounds(_np(q), _np(k), _np(v), _np(g), ok,
                                  d ** -0.5 if scale is None else scale, dtype)
    _close(out, *r["out"])
    got = _np(lse)
    assert np.array_equal(np.isneginf(got), np.isneginf(lse_ref))
    fin = np.isfinite(lse_ref)
    assert (np.abs(got[fin] - lse_ref[fin]) <= lse_tol[fin]).all()
    if backward:
        for name, x in zip(("dq", "dk", "dv"), grads):
            _close(x, *r[name])
    return out, lse, grads


SIZES = [  # b, nq, nk, h, kv, d
    (1, 1, 1, 1, 1, 8), (2, 1, 65, 4, 2, 64), (2, 3, 127, 2, 2, 128), (1, 128, 128, 2, 1, 64),
    (2, 129, 257, 4, 1, 128), (1, 300, 129, 2, 2, 80), (3, 17, 64, 6, 2, 96), (1, 260, 500, 1, 1, 40),
    (2, 64, 63, 3, 3, 36), (1, 33, 70, 2, 1, 33), (1, 5, 9, 2, 2, 1), (2, 16, 700, 2, 1, 128),
    (1, 9, 1500, 8, 1, 64), (1, 513, 385, 2, 1, 16), (4, 1, 300, 16, 4, 128), (2, 70, 130, 2, 2, 120)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", ["all", "len", "mask", "both"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", SIZES)
def test_attention(dtype, keys, b, nq, nk, h, kv, d):
    _check_attention(*_inputs(dtype, b, nq, nk, h, kv, d, keys))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", ["all", "len", "mask"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", [(1, 1, 4097, 1, 1, 64), (2, 5, 2500, 8, 2, 96),
                                            (1, 40, 1999, 1, 1, 128), (40, 1, 700, 8, 8, 32)])
def test_attention_few_rows_many_parts(dtype, keys, b, nq, nk, h, kv, d):
    """Parts of the key axis: one, a cluster's, more than a cluster's."""
    _check_attention(*_inputs(dtype, b, nq, nk, h, kv, d, keys), backward=False)


# more entries than one wave of blocks takes (they run in the order of their lengths), more
# entries than are ordered, and parts of a fixed length
@pytest.mark.parametrize("keys", ["len", "both"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", [(60, 1, 1030, 8, 4, 64), (128, 1, 600, 4, 4, 32),
                                            (130, 1, 600, 4, 4, 32), (12, 1, 4500, 4, 4, 64),
                                            (40, 3, 1100, 8, 4, 36)])
def test_attention_tokens_of_many_ragged_entries(keys, b, nq, nk, h, kv, d):
    q, k, v, g, kv_len, mask, ok = _inputs(BF16, b, nq, nk, h, kv, d, keys, seed=23)
    if keys == "len":   # equal lengths have an order too
        kv_len[b // 2:] = kv_len[b // 2].clone()
        ok = B.permitted(b, nk, kv_len.cpu().numpy(), None)
        bad = torch.from_numpy(~ok).cuda()
        k, v = (torch.nan_to_num(x.float(), nan=0.5, posinf=0.25).to(x.dtype) for x in (k, v))
        k[bad], v[bad] = float("nan"), float("inf")
    _check_attention(q, k, v, g, kv_len, mask, ok, backward=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq,h", [(1, 4), (70, 2)])
@pytest.mark.parametrize("nk", [40, 700, 1100])
def test_attention_masks_that_pad(dtype, nq, h, nk):
    """The mask permits the first keys of each entry: all, none, one, and ends at, before and
    behind a boundary of 16, 128 and 512 keys."""
    ends = sorted({min(e, nk) for e in (nk, 0, 1, 15, 16, 17, 127, 128, 129, 511, 512, 513, nk - 1)})
    b = len(ends)
    q, k, v, g, _, _, _ = _inputs(dtype, b, nq, nk, h, 2, 64, "all", seed=29)
    ok = np.arange(nk)[None, :] < np.array(ends)[:, None]
    mask = torch.from_numpy(ok.astype(np.uint8)).cuda()
    bad = torch.from_numpy(~ok).cuda()
    k[bad], v[bad] = float("nan"), float("inf")
    _check_attention(q, k, v, g, None, mask, ok)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("keys", ["all", "both"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", [(1, 20, 3100, 2, 1, 64), (1, 2500, 40, 2, 1, 128),
                                            (2, 700, 1100, 2, 1, 72), (1, 1, 2000, 3, 3, 33)])
def test_attention_gradients_in_parts(dtype, keys, b, nq, nk, h, kv, d):
    """Few blocks with long walks: the sums of dQ, or of dK and dV, come in parts."""
    _check_attention(*_inputs(dtype, b, nq, nk, h, kv, d, keys))


@pytest.mark.parametrize("d", [64, 128, 36])
@pytest.mark.parametrize("nk,few", [(2, 2), (7, 7), (130, 3), (700, 5), (128, 128), (129, 129)])
def test_attention_gradients_with_few_keys(d, nk, few):
    """bf16, few permitted keys (a short list, or all but a few masked): dS = P (dP - delta) is
    then of the size of out's own rounding times dout, so delta may not be taken from out.  A
    norm-wise check, relative to the gradients: P, dS and the result are rounded once each
    (u = 2^-8 at most each and 0.4 u in the root mean square, so 1.5 u holds three of them
    together with room)."""
    q, k, v, g, *_ = _inputs(BF16, 2, 90, nk, 4, 2, d, "all", seed=nk)
    mask = None
    if few < nk:
        mask = torch.zeros(2, nk, dtype=torch.uint8, device="cuda")
        at = torch.from_numpy(np.random.default_rng(few).permutation(nk)[:few]).cuda()
        mask[:, at] = 1
    ok = np.ones((2, nk), bool) if mask is None else _np(mask) != 0
    out, lse = K.cross_attention(q, k, v, key_mask=mask)
    got = K.cross_attention_backward(g, q, k, v, out, lse, key_mask=mask)
    ref = B.cross_attention_backward(_np(g), _np(q), _np(k), _np(v), ok)
    for x, y in zip(got, ref):
        assert np.linalg.norm(_np(x) - y) <= 3 * 2.0 ** -9 * np.linalg.norm(y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128, 36])
def test_attention_gradients_with_one_key_are_zero(dtype, d):
    """A softmax over one key is constant: dq and dk are exactly zero, dv is the sum of dout."""
    q, k, v, g, *_ = _inputs(dtype, 3, 150, 200, 2, 1, d, "all")
    mask = torch.ones(3, 200, dtype=torch.uint8, device="cuda")
    mask[1] = 0
    mask[1, 177] = 1
    for kv_len, m, b, at in ((torch.tensor([1, 5, 200], dtype=torch.int32, device="cuda"), None, 0, 0),
                             (None, mask, 1, 177)):
        out, lse = K.cross_attention(q, k, v, kv_len, m)
        dq, dk, dv = K.cross_attention_backward(g, q, k, v, out, lse, kv_len, m)
        assert (dq[b] == 0).all() and (dk[b] == 0).all()
        assert all((dq[i] != 0).any() for i in range(3) if i != b)
        want = _np(g[b]).sum(axis=(0, 1))
        got = _np(dv[b])
        assert (np.delete(got, at, axis=0) == 0).all()
        bound = np.abs(_np(g[b])).sum(axis=(0, 1)) * (SLACK + U[dtype] * (dtype == BF16)) + U[dtype] * np.abs(want)
        assert (np.abs(got[at, 0] - want) <= bound).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_without_queries_or_keys(dtype):
    q, k, v, g, *_ = _inputs(dtype, 2, 5, 7, 2, 2, 64, "all")
    out, lse = K.cross_attention(q, k[:, :0], v[:, :0])
    assert (out == 0).all() and torch.isneginf(lse).all()
    dq, dk, dv = K.cross_attention_backward(g, q, k[:, :0], v[:, :0], out, lse)
    assert (dq == 0).all() and dk.numel() == 0
    out, lse = K.cross_attention(q[:, :0], k, v)
    assert out.numel() == 0
    dk, dv = torch.full_like(k, 3), torch.full_like(v, 3)
    K.cross_attention_backward(g[:, :0], q[:, :0], k, v, out, lse, dk=dk, dv=dv)
    assert (dk == 0).all() and (dv == 0).all()
    K.cross_attention(q[:0], k[:0], v[:0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [3, 200])
def test_attention_large_scores_and_one_key(dtype, nq):
    """Scores of several hundred (a maximum that keeps growing along the keys) and rows with a
    single permitted key."""
    q, k, v, g, *_ = _inputs(dtype, 1, nq, 400, 2, 1, 64, "all")
    k = (k.float() * torch.linspace(0.1, 30, 400, device="cuda").view(1, -1, 1, 1)).to(dtype)
    _check_attention(q, k, v, g, None, None, B.permitted(1, 400))
    mask = torch.zeros(1, 400, dtype=torch.bool, device="cuda")
    mask[0, 257] = True
    _check_attention(q, k, v, g, None, mask, _np(mask) != 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq", [2, 150])
def test_attention_strides(dtype, nq):
    """Packed projections, heads before rows, one encoder for every batch entry (stride 0), rows
    that are not 16-byte aligned, and outputs within wider buffers."""
    b, nk, h, kv, d = 2, 190, 4, 2, 64
    q, k, v, g, kv_len, mask, ok = _inputs(dtype, b, nq, nk, h, kv, d, "len")
    k, v = k.nan_to_num(), v.nan_to_num(posinf=0)
    want = _check_attention(q, k, v, g, kv_len, mask, ok)
    packed = torch.zeros(b, nk, 2, kv, d + 8, device="cuda", dtype=dtype)
    pk, pv = packed[:, :, 0, :, :d], packed[:, :, 1, :, :d]
    pk.copy_(k), pv.copy_(v)
    hq = q.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.zeros(b, nq, h, d + 16, device="cuda", dtype=dtype)
    out, lse = K.cross_attention(hq, pk, pv, kv_len, out=wide[..., :d])
    dkv = torch.zeros_like(packed)
    grads = K.cross_attention_backward(g, hq, pk, pv, out, lse, kv_len, dk=dkv[:, :, 0, :, :d],
                                       dv=dkv[:, :, 1, :, :d])
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for x, y in zip(grads, want[2]):
        assert torch.equal(x, y)
    assert (wide[..., d:] == 0).all() and (dkv[..., d:] == 0).all()
    # rows that start at odd multiples of the element size
    odd = lambda t: torch.zeros(t.shape[0], t.shape[1], t.shape[2], t.shape[3] + 1, device="cuda",
                                dtype=dtype)[..., 1:].copy_(t)
    _check_attention(odd(q), odd(k), odd(v), odd(g), kv_len, mask, ok)
    # one encoder output read by every batch entry and head
    k1, v1 = k[:1, :, :1].expand(b, nk, kv, d), v[:1, :, :1].expand(b, nk, kv, d)
    _check_attention(q, k1, v1, g, kv_len, mask, ok)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_scale_other_stream_and_repeat(dtype):
    q, k, v, g, kv_len, mask, ok = _inputs(dtype, 2, 140, 333, 4, 2, 64, "both")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = _check_attention(q, k, v, g, kv_len, mask, ok, scale=0.3, stream=side)
    c = _check_attention(q, k, v, g, kv_len, mask, ok, scale=0.3, stream=side.cuda_stream)
    for x, y in zip((a[0], a[1], *a[2]), (c[0], c[1], *c[2])):
        assert torch.equal(x, y)   # no atomics: the same bits


@pytest.mark.parametrize("nq", [1, 130])
def test_attention_offsets_past_32_bits(nq):
    """Batch entries 2^31 elements apart, in k, v and their gradients."""
    b, nk, kv, d = 2, 150, 1, 64
    q, k, v, g, *_ = _inputs(BF16, b, nq, nk, 2, kv, d, "all")
    far = 2 ** 31 + 64

    def spread(t):
        big = torch.empty(far + nk * kv * d, device="cuda", dtype=BF16)
        y = big.as_strided((b, nk, kv, d), (far, kv * d, d, 1))
        return y.copy_(t)

    want = _check_attention(q, k, v, g, None, None, B.permitted(b, nk))
    fk, fv = spread(k), spread(v)
    out, lse = K.cross_attention(q, fk, fv)
    dk, dv = spread(torch.zeros_like(k)), spread(torch.zeros_like(v))
    dq, _, _ = K.cross_attention_backward(g, q, fk, fv, out, lse, dk=dk, dv=dv)
    for x, y in zip((out, lse, dq, dk, dv), (want[0], want[1], *want[2])):
        assert torch.equal(x, y)


def test_attention_gradient_is_a_difference_of_the_loss():
    """Along random directions, fp32: a central difference of sum(dout out) against <dx, direction>."""
    q, k, v, g, kv_len, mask, ok = _inputs(F32, 2, 20, 50, 4, 2, 32, "both")
    k, v = k.nan_to_num(), v.nan_to_num(posinf=0)
    out, lse = K.cross_attention(q, k, v, kv_len, mask)
    grads = K.cross_attention_backward(g, q, k, v, out, lse, kv_len, mask)
    loss = lambda a, b_, c: float((K.cross_attention(a, b_, c, kv_len, mask)[0].double() * g.double()).sum())
    h = 1e-2
    for i in range(3):
        e = _randn(50 + i, *(q, k, v)[i].shape)
        x = [q, k, v]
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + h * e, x[i] - h * e
        diff = (loss(*up) - loss(*down)) / (2 * h)
        dot = float((grads[i].double() * e.double()).sum())
        # truncation h^2/6 f''' (f''' of order |e|^3 per row, rows independent) and fp32 rounding / h
        size = float((grads[i].double().abs() * e.double().abs()).sum())
        assert abs(diff - dot) <= 5e-3 * size + 1e-3


def test_attention_refusals_of_the_python_layer():
    q, k, v, g, kv_len, mask, ok = _inputs(BF16, 2, 4, 6, 2, 2, 64, "both")
    with pytest.raises(ValueError):
        K.cross_attention(q, k.float(), v)
    with pytest.raises(ValueError):
        K.cross_attention(q, k, v[:, :3])
    with pytest.raises(ValueError):
        K.cross_attention(q, k, v, kv_len=kv_len.long())
    with pytest.raises(ValueError):
        K.cross_attention(q, k, v, key_mask=mask[:, :3])
    with pytest.raises(ValueError):
        K.cross_attention(q, k, v, lse=torch.empty(2, 4, 2, device="cuda"))
    with pytest.raises(ValueError):
        K.cross_attention(q.transpose(2, 3), k, v)
    with pytest.raises(K.KfacError, match="UNSUPPORTED"):
        x = torch.zeros(1, 2, 1, 136, device="cuda", dtype=BF16)
        K.cross_attention(x, x, x)
    out, lse = K.cross_attention(q, k, v, kv_len, mask)
    with pytest.raises(K.KfacError, match="WORKSPACE"):
        K.cross_attention_backward(g, q, k, v, out, lse, kv_len, mask,
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# one query tile per block with 64 and with 128 channels, two with 128, and the fp32 kernels
@pytest.mark.parametrize("size", [1.0, 1e30])
@pytest.mark.parametrize("dtype,d,nq", [(BF16, 64, 200), (BF16, 128, 100), (BF16, 128, 300),
                                        (BF16, 72, 300), (F32, 64, 100)])
def test_attention_scores_that_leap(dtype, d, nq, size):
    """A maximum that grows by 3 to 60 from one 64 keys to the next, in the first and in the second
    half of a 128-key tile, by other amounts in every row, and v of any size that 2^8 len_kv |v|
    keeps below 2^128: the weighted mean is finite, and so is out."""
    nk = 640
    q, k, v, g, *_ = _inputs(dtype, 1, nq, nk, 2, 1, d, "all", seed=31)
    steps = torch.tensor([0.0, 4, 60, 20, 27, 90, 93, 150, 156, 175], device="cuda")
    q[..., 0] = 8 * torch.linspace(0.05, 1, nq, device="cuda").view(1, -1, 1).to(dtype)
    k[..., 0] = (steps.repeat_interleave(64) * d ** 0.5 / 8).view(1, -1, 1).to(dtype)
    v = (size * v.float()).to(dtype)
    _check_attention(q, k, v, g, None, None, B.permitted(1, nk), backward=size == 1.0)


def _mean_error(got, ref):
    return float(((got.double() - ref) / ref).mean())


def _positive(seed, n, h, d):
    """Uniform in [1, 2) times a factor of each channel's own: means that are spread over a binade
    round to bf16 in both directions."""
    x = torch.rand(1, n, h, d, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    return ((1 + x) * 2 ** (torch.arange(h * d, device="cuda").view(h, d) / (h * d))).to(BF16)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_walks_along_the_keys(d):
    """524288 keys, v positive: what the tensor cores' accumulators lose to rounding towards zero
    would add up.  No sum of like signs is off by more than 2^-12 on average; P's and the
    result's roundings (2^-9 at most, of either sign, on 64 or more channels' means) average to a
    tenth of that or two, so 2^-11 holds both.
    dq, whose terms have both signs, in norm: P, dS and the result rounded once, and delta, which is
    taken from the rounded out: u sum_d |dout out| in every dS of a row."""
    nq, nk, h = 8192, 524288, 2
    q, k, g = (_randn(i, 1, n, h, d, dtype=BF16) for i, n in ((1, nq), (2, nk), (3, nq)))
    v = _positive(4, nk, h, d)
    out, lse = K.cross_attention(q, k, v)
    dq, _, _ = K.cross_attention_backward(g, q, k, v, out, lse)
    at = torch.arange(5, nq, 171, device="cuda")
    for j in range(h):
        Q, Kk, V, G = q[0, at, j].double(), k[0, :, j].double(), v[0, :, j].double(), g[0, at, j].double()
        p = torch.softmax(Q @ Kk.T * d ** -0.5, dim=-1)
        o = p @ V
        assert abs(_mean_error(out[0, at, j], o)) <= 2.0 ** -11
        dp = G @ V.T
        want = (p * (dp - (p * dp).sum(dim=-1, keepdim=True))) @ Kk * d ** -0.5
        of_delta = U[BF16] * (G * o).abs().sum(dim=-1, keepdim=True) * (p @ Kk) * d ** -0.5
        assert (dq[0, at, j].double() - want).norm() <= 3 * 2.0 ** -9 * want.norm() + of_delta.norm()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_walks_along_the_queries(d):
    """The same for dV, summed over 4 heads x 131072 queries, dout positive."""
    nq, nk, h = 131072, 9728, 4
    q, k, v = (_randn(i, 1, n, x, d, dtype=BF16) for i, n, x in ((1, nq, h), (2, nk, 1), (3, nk, 1)))
    g = _positive(4, nq, h, d)
    out, lse = K.cross_attention(q, k, v)
    _, _, dv = K.cross_attention_backward(g, q, k, v, out, lse)
    at = torch.arange(3, nk, 101, device="cuda")
    want = torch.zeros(len(at), d, device="cuda", dtype=torch.float64)
    for j in range(h):
        for x in range(0, nq, 16384):
            s = q[0, x:x + 16384, j].double() @ k[0, :, 0].double().T * d ** -0.5
            want += torch.softmax(s, dim=-1)[:, at].T @ g[0, x:x + 16384, j].double()
    assert abs(_mean_error(dv[0, at, 0], want)) <= 2.0 ** -11


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long_walks_of_single_tokens(d):
    """The same for out with one query per key head and more of them than blocks fit: one
    encoder's 1048576 states read by all."""
    b, nk, h = 64, 1048576, 8
    q, k, v = _randn(1, b, 1, h, d, dtype=BF16), _randn(2, 1, nk, 1, d, dtype=BF16), _positive(3, nk, 1, d)
    out, _ = K.cross_attention(q, k.expand(b, nk, h, d), v.expand(b, nk, h, d))
    p = torch.softmax(q[:8].view(-1, d).double() @ k.view(nk, d).double().T * d ** -0.5, dim=-1)
    assert abs(_mean_error(out[:8].view(-1, d), p @ v.view(nk, d).double())) <= 2.0 ** -11


def _owner(p):
    """The stream whose memory address p is in."""
    return next(x["stream"] for x in torch.cuda.memory_snapshot()
                if x["address"] <= p < x["address"] + x["total_size"])


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_and_workspaces_belong_to_the_given_stream(monkeypatch, raw):
    """Memory that torch's allocator takes back is handed out again at once to the stream it belongs
    to, before that stream's kernels have ended: what a call on another stream allocates has to be
    that stream's.  (Shown by ownership alone: nothing here depends on timing.)"""
    q, k, v, g, *_ = _inputs(BF16, 1, 20, 3100, 2, 1, 64, "all")
    table = K.rope_table(64, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    made, empty = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: made.append(empty(*a, **kw)) or made[-1])
    K.rope_table(64, 64, stream=stream)
    K.rope_table(64, 64, device="cuda", stream=stream)
    K.rope(q, q, table, stream=stream)
    K.dropout(q, 0.5, 1, stream=stream)
    K.dropout_backward(q, 0.5, 1, stream=stream)
    out, lse = K.cross_attention(q, k, v, stream=stream)
    K.cross_attention_backward(g, q, k, v, out, lse, stream=stream)
    side.synchronize()
    assert len(made) == 13 and all(t.numel() for t in made)
    assert {_owner(t.data_ptr()) for t in made} == {side.cuda_stream}
    made.clear()
    K.dropout(q, 0.5, 1)
    assert {_owner(t.data_ptr()) for t in made} == {torch.cuda.current_stream().cuda_stream}


def test_another_stream_leaves_memory_with_queued_readers_alone():
    """A tensor that was freed while its reader is queued, then calls on another stream that
    allocate as much."""
    n = 1 << 20
    z, side = torch.randn(n, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    x = torch.full((n,), 7.0, device="cuda")
    torch.cuda._sleep(200_000_000)   # about 0.1 s
    y = x + 1
    del x
    made = [K.dropout(z, 0.0, 1, stream=side) for _ in range(4)]
    torch.cuda.synchronize()
    assert (y == 8).all() and all(torch.equal(t, z) for t in made)


def test_attention_refuses_a_scale_of_zero():
    q, k, v, g, *_ = _inputs(BF16, 1, 4, 6, 2, 2, 64, "all")
    out, lse = K.cross_attention(q, k, v, scale=0.25)
    for call in (lambda s: K.cross_attention(q, k, v, scale=s),
                 lambda s: K.cross_attention_backward(g, q, k, v, out, lse, scale=s)):
        with pytest.raises(ValueError, match="scale"):
            call(0.0)
        with pytest.raises(K.KfacError):
            call(-0.25)


@pytest.mark.parametrize("keys", ["all", "both"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", [
    (1, 20, 3100, 2, 1, 64), (1, 2500, 40, 2, 1, 128), (2, 700, 1100, 2, 1, 72), (1, 1, 2000, 3, 3, 33),
    (2, 129, 257, 4, 1, 128), (1, 300, 129, 2, 2, 80), (1, 260, 500, 1, 1, 40), (1, 513, 385, 2, 1, 16),
    (2, 70, 130, 2, 2, 120), (3, 577, 1531, 4, 1, 64), (1, 900, 1400, 2, 2, 128)])
def test_attention_gradients_in_norm(keys, b, nq, nk, h, kv, d):
    """bf16 over several tiles and parts: the gradients as whole arrays, within what the roundings
    alone explain (a term or a tile that is missing does not fit: see the bounds' own test)."""
    q, k, v, g, kv_len, mask, ok = _inputs(BF16, b, nq, nk, h, kv, d, keys, seed=37)
    out, lse = K.cross_attention(q, k, v, kv_len, mask)
    got = K.cross_attention_backward(g, q, k, v, out, lse, kv_len, mask)
    ref, bound = B.gradient_norm_bounds(_np(g), _np(q), _np(k), _np(v), ok)
    for x, y, most in zip(got, ref, bound):
        assert np.linalg.norm(_np(x) - y) <= most


# the last sizes that the token kernel takes and the first that it does not, by heads per key head
@pytest.mark.parametrize("keys", ["all", "both"])
@pytest.mark.parametrize("b,nq,nk,h,kv,d", [
    (2, 16, 300, 2, 2, 64), (2, 17, 300, 2, 2, 64), (2, 8, 300, 4, 2, 96), (2, 9, 300, 4, 2, 96),
    (2, 12, 1030, 4, 1, 128), (2, 13, 1030, 4, 1, 128), (1, 12, 513, 16, 2, 32), (1, 13, 513, 16, 2, 32),
    (3, 12, 129, 16, 1, 128), (3, 13, 129, 16, 1, 128), (1, 12, 700, 32, 1, 64), (1, 13, 700, 32, 1, 64)])
def test_attention_few_queries_of_shared_key_heads(keys, b, nq, nk, h, kv, d):
    _check_attention(*_inputs(BF16, b, nq, nk, h, kv, d, keys, seed=41))
