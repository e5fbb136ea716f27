"""GPU parity of the operators of the parameters without Kronecker factors with the float64
reference: root-mean-square norms and the token embedding.

Tolerances, fixed before the first run.  u = 2^-8 bounds a rounding to bf16, f = 2^-24 one to fp32.
 * norms: a thread sums at most 64 squares in turn and the tree adds ten: a positive sum is within
   74 f, its root within 37 f, and y, r and the scales take a few more roundings: 64 f of |y|.  The
   result is rounded once.
 * dx: the same for the mean of w n (74 f of the mean of |w n|) and the products: 96 f of the terms'
   magnitudes.
 * sums over rows or tokens: f per term of the sum of magnitudes, and a few for the parts.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import second_order_optimizer_gb300 as K  # noqa: E402
from oracle import params_oracle as R  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
F = 2.0 ** -24


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


# -------------------------------------------------------------------------------------- norms

# every form: a warp, 256 and 1024 threads a row with one to eight vectors each, whole vectors and
# single elements, rows wider than registers hold
NORM_SIZES = [(1, 1), (3, 7), (5, 32), (9, 200), (17, 256), (4, 512), (33, 513), (16, 2048),
              (700, 1025), (2, 2056), (3, 4096), (2, 5001), (5, 8192), (2, 12000), (1, 20003), (3, 40000)]


def _check_norm(x, gain, res, eps, y, h, rstd):
    ref, s, r = R.rms_norm(_np(x), None if gain is None else _np(gain),
                           None if res is None else _np(res), eps)
    u = U[x.dtype]
    _close(y, ref, (u + 64 * F) * np.abs(ref))
    _close(rstd, r, 64 * F * r)
    if res is None:
        assert h is None
    else:
        _close(h, s, (u + F) * np.abs(s))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_norm(dtype, rows, cols):
    x, res = _randn(1, rows, cols, dtype=dtype), _randn(2, rows, cols, dtype=dtype)
    gain = 1 + 0.3 * _randn(3, cols)
    for g, r, eps in ((gain, res, 1e-6), (None, None, 0.5), (gain, None, 0.0)):
        y, h, rstd = K.rms_norm(x, g, r, eps)
        _check_norm(x, g, r, eps, y, h, rstd)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
@pytest.mark.parametrize("group", [0, 32, 128])
def test_norm_in_8_bits(dtype, rows, cols, group):
    x, res = _randn(1, rows, cols, dtype=dtype), _randn(2, rows, cols, dtype=dtype)
    x[0], res[0] = 0, 0                              # a row of zeros: scale 0, q 0
    gain = 1 + 0.3 * _randn(3, cols)
    q, scales, h = K.rms_norm_e4m3(x, gain, res, group=group)
    ref, s, _ = R.rms_norm(_np(x), _np(gain), _np(res))
    _, want = R.quantize(ref, group)
    _close(scales, want, 72 * F * want)
    _close(h, s, (U[dtype] + F) * np.abs(s))
    each = np.repeat(want, group or cols, axis=1)[:, :cols]
    # half a step of three mantissa bits, of the least exponent's step below 2^-6, and the division's
    # own roundings, which may turn a value near a border
    _close(q.float() * scales.repeat_interleave(group or cols, dim=1)[:, :cols], ref,
           (2.0 ** -4 + 200 * F) * np.abs(ref) + each * 2.0 ** -10)
    top = np.abs(_np(q.float()))
    for c in range(0, cols, group or cols):          # the largest of each group becomes 448
        assert (top[1:, c:c + (group or cols)].max(axis=1) == 448).all()


def test_norm_strides_in_place_and_shapes():
    rows, cols = 37, 96
    wide, other = _randn(1, rows, 200, dtype=BF16), _randn(2, rows, 128, dtype=BF16)
    x, res, gain = wide[:, 8:8 + cols], other[:, :cols], 1 + 0.1 * _randn(3, cols)
    want = K.rms_norm(x.contiguous(), gain, res.contiguous())
    out = torch.full((rows, 100), 7.0, device="cuda", dtype=BF16)
    y, h, _ = K.rms_norm(x, gain, res, out=out[:, 2:98])    # rows of 4-byte alignment
    assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    assert (out[:, :2] == 7).all() and (out[:, 98:] == 7).all()
    rest = wide[:, 8 + cols:].clone()
    y, h, _ = K.rms_norm(x, gain, res, residual_out=x)       # the stream over x
    assert torch.equal(y, want[0]) and torch.equal(x, want[1]) and torch.equal(wide[:, 8 + cols:], rest)
    x3 = _randn(4, 2, 3, 64)
    y, _, rstd = K.rms_norm(x3)
    assert y.shape == x3.shape and rstd.shape == (2, 3)
    y1, _, r1 = K.rms_norm(x3[0, 0])
    assert torch.equal(y1, y[0, 0]) and r1.shape == ()
    assert K.rms_norm(x3[:0])[0].shape == (0, 3, 64)


@pytest.mark.parametrize("cols", [40, 33, 3000, 30001])
def test_norm_in_place_over_the_residual(cols):
    x, res = _randn(1, 5, cols, dtype=BF16), _randn(2, 5, cols, dtype=BF16)
    want = K.rms_norm(x, None, res)
    got = K.rms_norm(x, None, res, residual_out=res)
    assert torch.equal(got[0], want[0]) and torch.equal(res, want[1])


def test_norm_of_extreme_rows():
    x = _randn(1, 5, 64)
    x[1] = 0
    x[2] *= 1e-18           # squares at the low end of fp32
    x[3, 5] = float("nan")
    x[4, 7] = float("inf")
    y, _, rstd = K.rms_norm(x, eps=1e-6)
    assert (y[1] == 0).all() and torch.allclose(rstd[1:3], torch.tensor(1e3, device="cuda"))
    assert torch.isnan(y[3]).all() and torch.isfinite(y[:3]).all()
    assert torch.isnan(y[4, 7]) and (y[4, :7] == 0).all()
    q, scales, _ = K.rms_norm_e4m3(x)
    assert torch.isnan(q[3].float()).all() and torch.isnan(scales[3:]).all() and (q[1].float() == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(9, 2), (33, 62), (40, 126), (17, 254), (40, 258), (9, 510),
                                       (5, 1022), (7, 2046), (3, 4094), (3, 4098), (2, 8190), (2, 8194)])
def test_norm_of_even_rows(dtype, rows, cols):
    """Rows of whole pairs, and the same rows where the pairs do not begin at whole words."""
    x, res, dy = (_randn(s, rows, cols, dtype=dtype) for s in (1, 2, 3))
    gain = 1 + 0.3 * _randn(4, cols)
    y, h, rstd = K.rms_norm(x, gain, res)
    _check_norm(x, gain, res, 1e-6, y, h, rstd)
    q, scales, _ = K.rms_norm_e4m3(x, gain, res, group=64)
    dx, dgain, square = K.rms_norm_backward(dy, h, gain, rstd, dresidual=res, square=True)
    ref = R.rms_norm_backward(_np(dy), _np(h), _np(gain), _np(rstd), _np(res))
    n, w = _np(h) * _np(rstd)[:, None], np.abs(_np(dy) * _np(gain))
    size = _np(rstd)[:, None] * (w + np.abs(n) * (w * np.abs(n)).mean(axis=1, keepdims=True))
    _close(dx, ref[0], 96 * F * (size + np.abs(_np(res))) + U[dtype] * np.abs(ref[0]))
    _close(dgain, ref[1], (rows + 16) * F * np.abs(_np(dy) * n).sum(axis=0))
    _close(square, ref[2], (rows + 20) * F * ref[2])
    odd = torch.empty(rows, cols + 1, device="cuda", dtype=dtype)[:, 1:]   # single elements
    odd.copy_(x)
    y1, h1, rstd1 = K.rms_norm(odd, gain, res)
    _check_norm(x, gain, res, 1e-6, y1, h1, rstd1)
    assert torch.equal(h1, h)
    q1, scales1, _ = K.rms_norm_e4m3(odd, gain, res, group=64)
    # (r's last bits move a scale by as much, and a value over it by no more than a step)
    _close(scales1, _np(scales), 128 * F * _np(scales))
    assert (q1.float() - q.float()).abs().le(q.float().abs() / 8 + 2.0 ** -9).all()


def test_norm_of_squares_beyond_fp32():
    """A sum of squares past 2^128 is taken as infinite: zeros; just below it the norm is exact."""
    x = torch.full((2, 64), 2.0**60, device="cuda")   # squares 2^120, their sum 2^126
    x[1, 3] = 2.0**64
    y, _, rstd = K.rms_norm(x, eps=0.0)
    assert torch.allclose(y[0], torch.ones(64, device="cuda"), rtol=1e-6) and (y[1] == 0).all()
    assert rstd[1] == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(5000, 64), (2500, 33)])
def test_norm_backward(dtype, rows, cols):
    h, dy, dh = (_randn(s, rows, cols, dtype=dtype) for s in (1, 2, 3))
    gain = 1 + 0.3 * _randn(4, cols)
    _, _, rstd = K.rms_norm(h, gain)
    for g, d in ((gain, dh), (None, None)):
        dx, dgain, square = K.rms_norm_backward(dy, h, g, rstd, dresidual=d, square=True)
        gn = None if g is None else _np(g)
        ref = R.rms_norm_backward(_np(dy), _np(h), gn, _np(rstd), None if d is None else _np(d))
        r, n = _np(rstd)[:, None], _np(h) * _np(rstd)[:, None]
        w = np.abs(_np(dy) * (1 if gn is None else gn))
        size = r * (w + np.abs(n) * (w * np.abs(n)).mean(axis=1, keepdims=True))
        size = size + (0 if d is None else np.abs(_np(d)))
        _close(dx, ref[0], 96 * F * size + U[dtype] * np.abs(ref[0]))
        each = np.abs(_np(dy) * n)
        _close(dgain, ref[1], (rows + 16) * F * each.sum(axis=0))
        _close(square, ref[2], (rows + 20) * F * ref[2])
        again = K.rms_norm_backward(dy, h, g, rstd, dresidual=d, square=True)
        assert torch.equal(dx, again[0]) and torch.equal(dgain, again[1]) and torch.equal(square, again[2])


def test_norm_backward_in_place_and_parts():
    h, dy, dh = (_randn(s, 50, 72, dtype=BF16) for s in (1, 2, 3))
    gain = 1 + 0.1 * _randn(4, 72)
    _, _, rstd = K.rms_norm(h, gain)
    ws = K.rms_norm_workspace(h)
    want = K.rms_norm_backward(dy, h, gain, rstd, dresidual=dh, workspace=ws)
    assert want[2] is None
    for over in (dy, dh):
        keep = over.clone()
        got = K.rms_norm_backward(dy, h, gain, rstd, dresidual=dh, dx=over, workspace=ws)
        assert torch.equal(over, want[0]) and torch.equal(got[1], want[1])
        over.copy_(keep)
    none = K.rms_norm_backward(dy[:0], h[:0], gain, rstd[:0], square=True)
    assert (none[1] == 0).all() and (none[2] == 0).all()


# ---------------------------------------------------------------------------------- embedding

EMBED_SIZES = [(1, 1, 1), (5, 10, 16), (1, 300, 40), (333, 7, 33), (1000, 5000, 520), (4097, 100, 65),
               (300, 40, 2), (17001, 700, 258), (260, 50, 1030), (2048, 70000, 72),
               (2049, 200, 72), (16384, 1000, 24),
               (16385, 70000, 8), (50000, 300, 16), (130, 1, 48), (20000, 3, 9)]


def _ids(seed, tokens, rows, kind, dtype):
    g = np.random.default_rng(seed)
    if kind == "hot":     # half the tokens on one row, the others uneven
        ids = np.minimum((rows * g.random(tokens) ** 3).astype(np.int64), rows - 1)
        ids[g.random(tokens) < 0.5] = rows // 2
    else:                 # some ids outside the table
        ids = g.integers(-2, rows + 2, tokens)
    return torch.from_numpy(ids).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,width", EMBED_SIZES)
def test_embedding(dtype, tokens, rows, width):
    table = _randn(1, rows, width, dtype=dtype)
    for id_type, scale in ((torch.int32, 1.0), (torch.int64, 5.5)):
        ids = _ids(2, tokens, rows, "any", id_type)
        got, ref = K.embedding(ids, table, scale), R.embedding(ids.cpu().numpy(), _np(table), scale)
        assert np.array_equal(np.isnan(_np(got)), np.isnan(ref))
        # the scale's rounding, the product's, the result's
        _close(torch.nan_to_num(got), np.nan_to_num(ref), (2 * F + U[dtype]) * np.abs(np.nan_to_num(ref)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,rows,width", EMBED_SIZES)
@pytest.mark.parametrize("kind", ["any", "hot"])
def test_embedding_backward(dtype, tokens, rows, width, kind):
    ids = _ids(3, tokens, rows, kind, torch.int64 if kind == "any" else torch.int32)
    dout = _randn(4, tokens, width, dtype=dtype)
    pad = 0 if kind == "any" else -1
    freq = torch.full((rows,), 9.0, device="cuda")
    ws = K.embedding_workspace(ids, rows, width)
    ws.fill_(255)         # whatever an earlier call left there
    got = K.embedding_backward(ids, dout, rows, 1.5, pad, frequency=freq, workspace=ws)
    at = ids.cpu().numpy()
    ref, want = R.embedding_backward(at, _np(dout), rows, 1.5, pad)
    size, _ = R.embedding_backward(at, np.abs(_np(dout)), rows, 1.5, pad)
    terms = np.round(want * tokens)[:, None] + 4
    _close(got, ref, terms * F * size)
    _close(freq, want, 2 * F * want)
    assert torch.equal(got, K.embedding_backward(ids, dout, rows, 1.5, pad))   # the same bits
    # added to what is there; rows without tokens keep even a NaN
    base = _randn(5, rows, width)
    base[torch.from_numpy(want == 0).cuda()] = float("nan")
    more = base.clone()
    K.embedding_backward(ids, dout, rows, 1.5, pad, out=more, accumulate=True, workspace=ws)
    none = (want == 0)
    assert np.isnan(_np(more)[none]).all()
    _close(more[~torch.from_numpy(none).cuda()], (ref + _np(base))[~none],
           (terms * F * size + F * np.abs(ref + _np(base)))[~none])


@pytest.mark.parametrize("width", [5, 16])
def test_embedding_backward_of_many_tokens_clears_the_other_rows(width):
    """Beyond one cluster's sort, whatever an earlier call left in the workspace: other ids, or anything."""
    tokens, rows = 16385, 40003
    dout = _randn(1, tokens, width)
    ws = None
    for seed, fill in ((2, 0), (3, None), (4, 255), (5, 1)):
        ids = _ids(seed, tokens, rows // seed, "any", torch.int64)
        ws = K.embedding_workspace(ids, rows, width) if ws is None else ws
        if fill is not None:
            ws.fill_(fill)
        store = torch.full((rows, width + 3), float("nan"), device="cuda")
        freq = torch.full((rows,), float("nan"), device="cuda")
        K.embedding_backward(ids, dout, rows, out=store[:, :width], frequency=freq, workspace=ws)
        ref, want = R.embedding_backward(ids.cpu().numpy(), _np(dout), rows, 1.0, -1)
        size, _ = R.embedding_backward(ids.cpu().numpy(), np.abs(_np(dout)), rows, 1.0, -1)
        _close(store[:, :width], ref, (np.round(want * tokens)[:, None] + 4) * F * size)
        _close(freq, want, 2 * F * want)
        assert torch.isnan(store[:, width:]).all()
        again = torch.full((rows,), float("nan"), device="cuda")   # frequencies alone are cleared
        K.embedding_backward(ids, dout, rows, out=store[:, :width], accumulate=True, frequency=again,
                             workspace=ws)
        assert torch.equal(again, freq)


@pytest.mark.parametrize("tokens", [100, 17000])
def test_embedding_backward_of_a_huge_table(tokens):
    """Ids of more than 24 bits: four passes of the sort."""
    rows = 2 ** 24 + 5
    ids = torch.from_numpy(np.random.default_rng(1).integers(rows - 300, rows + 3, tokens)).cuda()
    dout = _randn(2, tokens, 1)
    got = K.embedding_backward(ids, dout, rows)
    ref, _ = R.embedding_backward(ids.cpu().numpy() - (rows - 300), _np(dout), 300)
    size, _ = R.embedding_backward(ids.cpu().numpy() - (rows - 300), np.abs(_np(dout)), 300)
    assert (got[:-300] == 0).all()
    _close(got[-300:], ref, 200 * F * size)


def test_embedding_strides_and_shapes():
    rows, width = 50, 24
    wide = _randn(1, rows, 40, dtype=BF16)
    table = wide[:, 8:32]
    ids = torch.randint(0, rows, (3, 7), device="cuda")
    want = K.embedding(ids, table.contiguous(), 2.0)
    assert want.shape == (3, 7, width) and torch.equal(K.embedding(ids, table, 2.0), want)
    out = torch.zeros(21, 30, device="cuda", dtype=BF16)
    K.embedding(ids.view(-1), table, 2.0, out=out[:, 3:27])
    assert torch.equal(out[:, 3:27], want.view(21, width)) and (out[:, 27:] == 0).all()
    dout = _randn(2, 21, 40, dtype=BF16)
    big = torch.full((rows, 30), 3.0, device="cuda")
    K.embedding_backward(ids.view(-1), dout[:, 8:32], rows, out=big[:, 1:25])
    assert torch.equal(big[:, 1:25], K.embedding_backward(ids.view(-1), dout[:, 8:32].contiguous(), rows))
    assert (big[:, 0] == 3).all() and (big[:, 25:] == 3).all()
    none = K.embedding_backward(ids[:0], dout.view(-1)[:0].view(0, 7, 40), rows)
    assert none.shape == (rows, 40) and (none == 0).all()
    with pytest.raises(ValueError, match="given out"):
        K.embedding_backward(ids.view(-1), dout, rows, accumulate=True)


def test_streams_and_graphs():
    """On another stream, and captured: two graphs with workspaces of their own, replayed in turn."""
    ids = _ids(3, 700, 90, "hot", torch.int64)
    dout, x, gain = _randn(1, 700, 64, dtype=BF16), _randn(2, 700, 64, dtype=BF16), _randn(3, 64)
    want = K.embedding_backward(ids, dout, 90)
    y, _, rstd = K.rms_norm(x, gain)
    grads = K.rms_norm_backward(dout, x, gain, rstd, square=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = K.embedding_backward(ids, dout, 90, stream=side)
    y2, _, r2 = K.rms_norm(x, gain, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(y2, y)
    graphs = []
    for _ in range(2):
        out = torch.empty_like(want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.embedding_backward(ids, dout, 90, out=out)
            gr = K.rms_norm_backward(dout, x, gain, rstd, square=True)
        graphs.append((g, out, gr))
    for _ in range(3):
        for g, out, gr in graphs:
            out.fill_(5)
            g.replay()
    for _, out, gr in graphs:
        assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(gr, grads))


@pytest.mark.parametrize("tokens", [7753, 16385])
def test_embedding_workspace_kept_for_the_largest_batch(tokens):
    """One token fewer may take more chunks: the kept workspace serves it all the same."""
    rows, width = 50021, 2048
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    ids = torch.randint(0, rows, (tokens,), generator=g, device="cuda")
    dout = torch.randn(tokens, width, generator=g, device="cuda").bfloat16()
    work = K.embedding_workspace(ids, rows, width)
    for n in (tokens, tokens - 1, tokens - 2, 5000, 17, 1, 0):
        got = K.embedding_backward(ids[:n], dout[:n], rows, workspace=work)
        # at most a dozen tokens of one id: sums of 12 values, 2^-24 of each partial sum
        want = torch.zeros(rows, width, device="cuda", dtype=torch.float64).index_add_(0, ids[:n], dout[:n].double())
        size = torch.zeros(rows, width, device="cuda", dtype=torch.float64).index_add_(0, ids[:n], dout[:n].double().abs())
        assert ((got - want).abs() <= 12 * 2.0 ** -24 * size).all(), n


def test_padding_ids_no_c_type_holds_are_refused():
    ids, dout = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(3, 8, device="cuda")
    for padding in (2**64 - 1, 2**64 + 5):    # not -1, not 5
        with pytest.raises(ValueError, match="padding_id"):
            K.embedding_backward(ids, dout, 9, padding_id=padding)
    with pytest.raises(K.KfacError, match="INVALID_ARG"):
        K.embedding_backward(ids, dout, 9, padding_id=-2)


def test_norm_workspace_of_a_scalar_is_refused():
    with pytest.raises(ValueError, match="channels"):
        K.rms_norm_workspace(torch.zeros((), device="cuda"))
