"""CPU checks of the operators of the parameters without Kronecker factors: the float64 reference
against what its definitions fix, and every refusal of the entry points that needs no GPU."""
import ctypes

import numpy as np
import pytest

from oracle import kfac_oracle as O
from oracle import params_oracle as R


# ------------------------------------------------------------------------------- the oracle

def _difference(loss, x, i, h=1e-5):
    """Central difference of loss() in x[i]: truncation h^2 and rounding 1e-16 / h, both about 1e-10."""
    keep = x[i]
    x[i] = keep + h
    up = loss()
    x[i] = keep - h
    down = loss()
    x[i] = keep
    return (up - down) / (2 * h)


def test_norm_gradients_are_differences_of_the_loss():
    rng = np.random.default_rng(0)
    x, res, gain = rng.standard_normal((5, 7)), rng.standard_normal((5, 7)), rng.standard_normal(7)
    g, gs = rng.standard_normal((5, 7)), rng.standard_normal((5, 7))

    def loss():   # the norm's output and the residual stream's other reader
        y, s, _ = R.rms_norm(x, gain, res, eps=0.1)
        return (y * g).sum() + (s * gs).sum()

    _, s, r = R.rms_norm(x, gain, res, eps=0.1)
    dx, dgain, square = R.rms_norm_backward(g, s, gain, r, gs)
    for k in range(12):
        i = tuple(rng.integers(0, n) for n in x.shape)
        assert abs(_difference(loss, x, i) - dx[i]) <= 1e-8
        assert abs(_difference(loss, res, i) - dx[i]) <= 1e-8
    for c in range(7):
        assert abs(_difference(loss, gain, (c,)) - dgain[c]) <= 1e-8
    each = g * s * r[:, None]
    assert np.allclose(square, O.diag_factor(each))   # the diagonal factor of the gain's gradients


def test_norm_of_a_row_has_mean_square_one():
    y, _, _ = R.rms_norm(np.random.default_rng(1).standard_normal((3, 50)) * 7, eps=0.0)
    assert np.allclose((y * y).mean(axis=1), 1)


def test_e4m3_is_the_formats_own_rounding():
    torch = pytest.importorskip("torch")
    v = np.concatenate([np.linspace(-448, 448, 20001), 2.0 ** np.arange(-12, 9), [0.0, 1e-4, 460.0]])
    v = v.astype(np.float32)
    want = torch.from_numpy(np.clip(v, -448, 448)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3(v), want)


@pytest.mark.parametrize("group", [0, 32])
def test_quantized_rows_are_within_half_a_step(group):
    y = np.random.default_rng(2).standard_normal((4, 70)) * 3
    y[1, 32:64] = 0
    q, scales = R.quantize(y, group)
    s = np.repeat(scales, group or 70, axis=1)[:, :70]
    assert (np.abs(q * s - y) <= 2.0 ** -4 * np.abs(y) + s * 2.0 ** -10).all()
    assert (np.abs(q).max() == 448) and (q[1, 32:64] == 0).all()


def test_embedding_gradient_is_the_transpose_of_the_lookup():
    rng = np.random.default_rng(3)
    table, ids = rng.standard_normal((6, 4)), np.array([[1, 5, 1], [0, 6, -2]])
    out = R.embedding(ids, table, 1.5)
    assert np.isnan(out[1, 1:]).all() and np.allclose(out[0, 1], 1.5 * table[5])
    dout = rng.standard_normal(out.shape)
    dt, freq = R.embedding_backward(ids, dout, 6, 1.5)
    assert np.isclose((dt * table).sum(), np.nansum(np.where(np.isnan(out), 0, out) * dout))
    assert np.allclose(freq, np.array([1, 2, 0, 0, 0, 1]) / 6)
    # the frequencies are the diagonal of the factor of the one-hot inputs
    hot = np.eye(7)[np.where((ids >= 0) & (ids < 6), ids, 6).reshape(-1)][:, :6]
    assert np.allclose(freq, O.diag_factor(hot))
    assert (R.embedding_backward(ids, dout, 6, 1.5, padding_id=1)[0][1] == 0).all()


def test_orthogonalize_is_the_newton_schulz_iteration():
    rng = np.random.default_rng(4)
    for shape in ((5, 9), (9, 5), (6, 6), (1, 7)):
        x = rng.standard_normal(shape)
        assert np.allclose(R.orthogonalize(x), R.newton_schulz(x), atol=1e-10)
        t = np.linalg.svd(R.orthogonalize(x), compute_uv=False)
        assert t.max() < 1.21 and np.allclose(R.orthogonalize(x), R.orthogonalize(5 * x), atol=1e-6)
    # the classic coefficients converge to the orthogonal factor itself
    x = rng.standard_normal((4, 8))
    u, _, vt = np.linalg.svd(x, full_matrices=False)
    assert np.allclose(R.orthogonalize(x, 30, (1.5, -0.5, 0.0)), u @ vt)
    assert (R.orthogonalize(np.zeros((3, 4))) == 0).all()


def test_orthogonal_step_by_hand():
    """One singular value: the direction is a multiple of the update."""
    g, m, w = np.array([[3.0, 4.0]]), np.array([[1.0, 0.0]]), np.array([[1.0, 2.0]])
    m1, w1 = R.orthogonal_step(g, m, w, 0.1, momentum=0.5, weight_decay=0.2, nesterov=False, steps=1,
                               coefficients=(2.0, -1.0, 0.0), eps=0.0)
    assert np.allclose(m1, [[3.5, 4.0]])                     # of norm t: 2 t - t^3 at t = 1 is 1
    assert np.allclose(w1, w - 0.1 * (m1 / np.sqrt(28.25) + 0.2 * w))


# ------------------------------------------------------------- refusals (nothing is launched)

@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import second_order_optimizer_gb300._lib as L
    return L


A, W, U = 1, 2, 7   # KFAC_ERR_INVALID_ARG, KFAC_ERR_WORKSPACE, KFAC_ERR_UNSUPPORTED
P = 0x10000         # an aligned address that is never read


def _norm(lib, x=P, res=None, gain=P, h=None, y=2 * P, rstd=P, q=None, scales=None, **kw):
    d = dict(dtype=1, rows=4, cols=16, eps=1e-6, ldx=16, ldr=16, ldh=16, ldy=16, ldq=16, group=0)
    d.update(kw)
    return lib.LIB.kfac_rms_norm(lib.NORM_DESC.pack(*d.values()), x, res, gain, h, y, rstd, q, scales,
                                 None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(rows=-1), dict(cols=-1), dict(eps=-1e-9), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(group=16), dict(group=-32), dict(x=None), dict(y=None),
    dict(x=P + 1), dict(y=P + 1), dict(gain=P + 2), dict(rstd=P + 2), dict(h=P + 1), dict(res=P + 1),
    dict(ldx=15), dict(ldy=-16), dict(res=3 * P, ldr=8), dict(h=3 * P, ldh=0),
    dict(q=P), dict(q=P, scales=P + 2), dict(q=P, scales=P, ldq=15),
    dict(h=P, ldh=32),                 # in place with another leading dimension
    dict(y=P), dict(h=2 * P)])         # the result over an input, two results in one place
def test_norm_refuses(lib, kw):
    assert _norm(lib, **kw) == A


def test_norm_limits(lib):
    assert _norm(lib, rows=0, x=None) == 0 and _norm(lib, cols=0, x=None) == 0
    big = dict(ldx=1 << 21, ldy=1 << 21, ldq=1 << 21)
    assert _norm(lib, cols=(1 << 20) + 1, **big) == U
    assert _norm(lib, cols=1 << 20, q=P, scales=P, group=32, **big) == U
    assert _norm(lib, rows=1 << 31) == U


def _norm_grad(lib, dy=P, h=P, gain=P, rstd=P, dh=None, dx=2 * P, dg=P, sq=P, ws=P, nb=1 << 30, **kw):
    d = dict(dtype=1, rows=4, cols=16, lddy=16, ldh=16, lddh=16, lddx=16)
    d.update(kw)
    return lib.LIB.kfac_rms_norm_backward(lib.NORM_GRAD_DESC.pack(*d.values()), dy, h, gain, rstd, dh,
                                          dx, dg, sq, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(rows=-1), dict(cols=-2), dict(dy=None), dict(h=None), dict(rstd=None),
    dict(dy=P + 1), dict(h=P + 1), dict(gain=P + 1), dict(rstd=P + 2), dict(dh=P + 1), dict(dx=P + 1),
    dict(dg=P + 2), dict(sq=P + 1), dict(lddy=15), dict(ldh=-1), dict(dh=3 * P, lddh=1), dict(lddx=4),
    dict(dx=P, lddx=32), dict(h=3 * P, dx=3 * P)])
def test_norm_backward_refuses(lib, kw):
    assert _norm_grad(lib, **kw) == A


def test_norm_backward_workspace(lib):
    n = ctypes.c_size_t(0)
    f = lib.LIB.kfac_rms_norm_workspace_size
    assert f(100, 24, ctypes.byref(n)) == 0 and n.value % 256 == 0 and n.value >= 2 * 24 * 4
    assert f(-1, 24, ctypes.byref(n)) == A and f(1, 24, None) == A
    assert f(1, (1 << 20) + 1, ctypes.byref(n)) == U
    assert [_norm_grad(lib, ws=None), _norm_grad(lib, ws=P + 64), _norm_grad(lib, nb=128)] == [W] * 3
    assert _norm_grad(lib, cols=0, dy=None) == 0
    assert _norm_grad(lib, rows=0, dg=None, sq=None, dy=None) == 0


def _embed(lib, ids=P, table=P, out=P, **kw):
    d = dict(dtype=1, id_bits=32, tokens=8, rows=10, width=16, scale=1.0, ldt=16, ldo=16)
    d.update(kw)
    return lib.LIB.kfac_embedding(lib.EMBEDDING_DESC.pack(*d.values()), ids, table, out, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(id_bits=16), dict(tokens=-1), dict(rows=-1), dict(width=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(ids=None), dict(ids=P + 2),
    dict(ids=P + 4, id_bits=64), dict(table=None), dict(table=P + 1), dict(out=None), dict(out=P + 1),
    dict(ldt=15), dict(ldo=-1)])
def test_embedding_refuses(lib, kw):
    assert _embed(lib, **kw) == A


def test_embedding_refuses_a_scale_beyond_fp32(lib):
    assert _embed(lib, scale=1e39) == A and _embed_grad(lib, scale=-1e39) == A
    assert _embed(lib, scale=3e38, tokens=0) == 0


def test_embedding_limits(lib):
    assert _embed(lib, tokens=0, ids=None) == 0 and _embed(lib, width=0, ids=None) == 0
    assert _embed(lib, tokens=1 << 31) == U and _embed(lib, rows=1 << 31) == U


def _embed_grad(lib, ids=P, dout=P, dt=P, pad=-1, acc=0, freq=None, ws=P, nb=1 << 30, **kw):
    d = dict(dtype=1, id_bits=64, tokens=8, rows=10, width=16, scale=1.0, ldt=16, ldo=16)
    d.update(kw)
    return lib.LIB.kfac_embedding_backward(lib.EMBEDDING_DESC.pack(*d.values()), ids, dout, dt, pad, acc,
                                           freq, ws, nb, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(id_bits=8), dict(tokens=-1), dict(scale=float("-inf")), dict(acc=2),
    dict(pad=-2), dict(freq=P + 2), dict(ids=None), dict(ids=P + 4), dict(dout=None), dict(dout=P + 1),
    dict(dt=None), dict(dt=P + 2), dict(ldt=8), dict(ldo=3)])
def test_embedding_backward_refuses(lib, kw):
    assert _embed_grad(lib, **kw) == A


def test_embedding_backward_workspace(lib):
    n = ctypes.c_size_t(0)
    f = lib.LIB.kfac_embedding_workspace_size
    assert f(8, 10, 16, ctypes.byref(n)) == 0 and n.value % 256 == 0 and n.value >= 2 * 8 * 4 + 2 * 10 * 4
    assert f(8, 10, 16, None) == A and f(-8, 10, 16, ctypes.byref(n)) == A
    assert [_embed_grad(lib, ws=None), _embed_grad(lib, ws=P + 16), _embed_grad(lib, nb=256)] == [W] * 3
    assert _embed_grad(lib, rows=0, dt=None) == 0 and _embed_grad(lib, width=0, dt=None) == 0


def test_python_refuses_cpu_tensors_and_wrong_types(lib):
    torch = pytest.importorskip("torch")
    import second_order_optimizer_gb300 as K
    x = torch.zeros(4, 16)
    for f in (lambda: K.rms_norm(x), lambda: K.rms_norm_e4m3(x), lambda: K.rms_norm_workspace(x),
              lambda: K.rms_norm_backward(x, x, None, x[:, 0]),
              lambda: K.embedding(torch.zeros(3, dtype=torch.int64), x),
              lambda: K.embedding_backward(torch.zeros(3, dtype=torch.int64), x[:3], 9)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        K.rms_norm(x.half())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        K.embedding(torch.zeros(3, dtype=torch.int64), x.double())


def _ortho(lib, rows=(8, 4), cols=(4, 4), x=None, ldx=(4, 4), out=None, ldo=(4, 4), ws=P, nb=1 << 30,
           coefficients=None, hp=None, m=None, step=False, count=None, **kw):
    d = dict(dtype=1, math=1, steps=5, eps=1e-7)
    d.update(kw)
    co = None if coefficients is None else (ctypes.c_double * len(coefficients))(*coefficients)
    desc = lib.ORTHO_DESC.pack(*d.values(), 0 if co is None else ctypes.addressof(co))
    n = len(rows)
    ints = lambda v: (ctypes.c_int * n)(*v)
    ptrs = lambda v, e: (ctypes.c_void_p * n)(*(v or [e + 4096 * i for i in range(n)]))
    i64 = lambda v: (ctypes.c_int64 * n)(*v)
    count = n if count is None else count
    if step:
        hp = dict(lr=0.1, momentum=0.9, decay=0.0, scale=1.0, nesterov=1, **{}) | (hp or {})
        return lib.LIB.kfac_orthogonal_step(desc, lib.ORTHO_STEP.pack(*hp.values()), count, ints(rows),
                                            ints(cols), ptrs(x, P), i64(ldx), ptrs(m, 2 * P), i64(ldx),
                                            ptrs(out, 3 * P), i64(ldo), ws, nb, None)
    return lib.LIB.kfac_orthogonalize(desc, count, ints(rows), ints(cols), ptrs(x, P), i64(ldx),
                                      ptrs(out, 3 * P), i64(ldo), ws, nb, None)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(math=2), dict(steps=0), dict(steps=33), dict(eps=-1.0), dict(eps=float("nan")),
    dict(rows=(8, -1)), dict(cols=(-4, 4)), dict(count=-1), dict(x=(P, None)), dict(x=(P + 1, P)),
    dict(out=(None, P)), dict(out=(P, P + 1)), dict(out=(5 * P, 5 * P)), dict(ldx=(3, 4)), dict(ldo=(4, -4)),
    dict(steps=1, coefficients=(float("nan"), 0, 0)), dict(steps=1, coefficients=(0.0, 0.0, 0.0)),
    dict(steps=2, coefficients=(1e5, 0, 0, 1e5, 0, 0)), dict(steps=1, coefficients=(1e9, 0, 0))])
def test_orthogonalize_refuses(lib, kw, step):
    assert _ortho(lib, step=step, **kw) == A


def test_orthogonal_step_refuses(lib):
    bad = [dict(lr=float("nan")), dict(momentum=float("inf")), dict(decay=float("nan")),
           dict(scale=float("inf")), dict(nesterov=2)]
    assert [_ortho(lib, step=True, hp=h) for h in bad] == [A] * len(bad)
    assert _ortho(lib, step=True, m=(P, None)) == A and _ortho(lib, step=True, m=(P, P + 2)) == A
    assert _ortho(lib, step=True, m=(P, P)) == A


def test_orthogonalize_limits_and_workspace(lib):
    assert _ortho(lib, count=0) == 0 and _ortho(lib, step=True, count=0) == 0
    assert _ortho(lib, rows=(0, 5), cols=(3, 0), x=(None, None), ws=None) == 0   # nothing to do
    assert _ortho(lib, rows=(32769, 4)) == U
    big = dict(rows=(200, 4), cols=(300, 4), ldx=(300, 4), ldo=(300, 4))
    assert [_ortho(lib, ws=None, **big), _ortho(lib, ws=P + 128, **big), _ortho(lib, nb=512, **big)] == [W] * 3
    n = ctypes.c_size_t(0)
    one = (ctypes.c_int * 1)
    size = lambda math, r, c: (lib.LIB.kfac_orthogonalize_workspace_size(
        lib.ORTHO_DESC.pack(1, math, 5, 0.0, 0), 1, one(r), one(c), ctypes.byref(n)), n.value)
    assert size(1, 200, 300)[0] == 0 and size(1, 200, 300)[1] % 256 == 0
    assert size(1, 200, 300)[1] >= 4 * 200 * 300 + 4 * 200 * 200
    assert size(0, 200, 300)[1] >= 2 * (4 * 200 * 300 + 4 * 200 * 200)
    assert size(1, 1024, 4096)[1] >= 4 * 1024 * 4096 + 10 * 1024 * 1024   # steps in groups
    assert size(1, 0, 300) == (0, 0) and size(1, 128, 300) == (0, 0)      # (in shared memory)
    assert size(1, 128, 4097)[1] > 0 and size(0, 1537, 128)[1] > 0
    assert lib.LIB.kfac_orthogonalize_workspace_size(lib.ORTHO_DESC.pack(1, 0, 5, 0.0, 0), 1, one(1),
                                                     one(1), None) == A


def test_python_refuses_matrices_that_do_not_fit(lib):
    torch = pytest.importorskip("torch")
    import second_order_optimizer_gb300 as K
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="CUDA"):
        K.orthogonalize(x)
    with pytest.raises(ValueError, match="rows, columns"):
        K.orthogonalize(x[0])
    from second_order_optimizer_gb300 import _params
    with pytest.raises(ValueError, match="triple"):
        _params._ortho_desc("orthogonalize", 0, None, 3, 0.0, [(1, 2, 3), (1, 2, 3)])
    desc, flat = _params._ortho_desc("orthogonalize", 0, None, 2, 0.0, (1.5, -0.5, 0))
    assert list(flat) == [1.5, -0.5, 0, 1.5, -0.5, 0]


@pytest.mark.parametrize("width", [1, 80, 512, 513, 2048, 8191, 1 << 20])
def test_embedding_workspace_serves_smaller_calls(lib, width):
    n = ctypes.c_size_t(0)

    def size(tokens, rows=50021):
        assert lib.LIB.kfac_embedding_workspace_size(tokens, rows, width, ctypes.byref(n)) == 0
        return n.value

    most = 0
    for tokens in [*range(1, 40), *range(7600, 7800), *range(16000, 16500, 3), *range(50000, 50600, 7), 1 << 20]:
        assert size(tokens) >= most, tokens
        most = size(tokens)
        assert size(tokens, 50020) <= most


def test_orthogonalize_workspace_serves_any_of_its_matrices(lib):
    """Small matrices need none in a launch of their own, but some beside large ones: what is kept for
    all of a list is enough for a part of it."""
    rng = np.random.default_rng(0)
    n = ctypes.c_size_t(0)

    def size(shapes, math, steps):
        ints = lambda v: (ctypes.c_int * len(shapes))(*v)
        assert lib.LIB.kfac_orthogonalize_workspace_size(
            lib.ORTHO_DESC.pack(1, math, steps, 0.0, 0), len(shapes), ints([s[0] for s in shapes]),
            ints([s[1] for s in shapes]), ctypes.byref(n)) == 0
        return n.value

    for math in (0, 1):
        shapes = [(64, 64)] * 30 + [(300, 200)]
        assert size(shapes, math, 5) >= size(shapes[20:], math, 5) > 0
        for _ in range(200):
            shapes = [tuple(int(v) for v in rng.integers(0, 200, 2)) for _ in range(rng.integers(1, 70))]
            shapes += [(int(rng.integers(129, 2000)), 1600) for _ in range(rng.integers(0, 5))]
            if rng.random() < 0.2:
                shapes += [(140, 150)] * int(rng.integers(10, 60))
            some = [s for s in shapes if rng.random() < rng.choice([0.2, 0.5, 0.9])]
            assert size(some, math, 5) <= size(shapes, math, 5)
            assert size(shapes, math, 1) <= size(shapes, math, 5)
    assert size([(64, 64)] * 40, 1, 5) == 0    # nothing for them to ride with


def test_embedding_backward_refuses_frequencies_of_rows_without_channels(lib):
    """(They would be left unwritten.)"""
    assert _embed_grad(lib, width=0, dt=None, freq=P) == A
    assert _embed_grad(lib, width=0, dt=None) == 0 and _embed_grad(lib, rows=0, width=0, dt=None, freq=P) == 0


def test_orthogonalize_refuses_results_over_other_inputs(lib):
    """In place is the same matrix with the same leading dimension; anything else would be read while it
    is written."""
    assert _ortho(lib, x=(P, 2 * P), out=(P, 5 * P), ldx=(4, 4), ldo=(8, 4)) == A     # another layout
    assert _ortho(lib, x=(P, 2 * P), out=(2 * P, P)) == A                             # each other's
    assert _ortho(lib, x=(P, P), out=(P, 5 * P)) == A                                 # x of the second as well
    step = lambda **kw: _ortho(lib, step=True, **kw)
    assert step(x=(P, 2 * P), m=(P, 6 * P)) == A and step(x=(P, 2 * P), out=(7 * P, P)) == A
    assert step(m=(7 * P, 8 * P), out=(8 * P, 9 * P)) == A and step(m=(7 * P, 8 * P), out=(7 * P, 9 * P)) == A
    # (these pass the checks: the next one, of the workspace, refuses)
    big = dict(rows=(200, 4), cols=(300, 4), ldx=(300, 4), ldo=(300, 4), ws=None)
    assert _ortho(lib, x=(P, 2 * P), out=(P, 2 * P), **big) == W
    assert _ortho(lib, x=(P, P), out=(5 * P, 6 * P), **big) == W
    assert _ortho(lib, x=(P, 2 * P), out=(P, 2 * P), **(big | dict(rows=(1, 200), cols=(4, 300), ldx=(4, 300), ldo=(9, 300)))) == W
    assert step(**big) == W


def test_what_fp32_does_not_hold_is_refused(lib):
    """eps that becomes infinite (results of 0) or zero (rows of zeros become NaN) as fp32; rates and
    decays of the step likewise."""
    assert _norm(lib, eps=1e39) == A and _norm(lib, eps=1e-46) == A
    assert [_norm(lib, eps=e, rows=0) for e in (0.0, 1e-45, 1e-12, 3e38)] == [0] * 4
    big = dict(rows=(200, 4), cols=(300, 4), ldx=(300, 4), ldo=(300, 4), ws=None)
    for hp in (dict(lr=1e39), dict(lr=1e30, scale=1e9), dict(momentum=1e39), dict(lr=1e20, decay=1e20),
               dict(lr=3e37)):   # times sqrt(32000 / 140) = 15.1
        assert _ortho(lib, step=True, hp=hp, **(big | dict(rows=(32000, 4), cols=(140, 4)))) == A
    assert _ortho(lib, step=True, hp=dict(lr=1e36), **big) == W   # (the next check)
