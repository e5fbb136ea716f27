"""GPU parity of the orthogonalised updates with the float64 reference.

Tolerances in norm, fixed before the first run.  Half arithmetic stores every matrix between the
products in fp16: the reference's own iteration with those roundings (newton_schulz_fp16) is e off,
and the kernel, whose roundings are as large but its own, may be 1.5 e off, and the result's rounding:
u = 2^-8 for bf16.  Full arithmetic stores 22 bits and sums at most 24 truncated terms per fp32
accumulator (24 2^-23 < 2^-18.4), 2^-19 where fp16 has 2^-11: e 2^-8, and 2^-24 for the result.
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
FULL, HALF = K.KFAC_ORTHO_FULL, K.KFAC_ORTHO_HALF
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def _np(t):
    return t.detach().double().cpu().numpy()


def _gradient(seed, rows, cols, dtype=F32, size=1e-4):
    """A few strong directions and noise."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    r = max(1, min(rows, cols) // 8)
    strong = torch.logspace(0, -1, r, device="cuda")
    return (size * ((randn(rows, r) * strong) @ randn(r, cols) / r ** 0.5 + 0.2 * randn(rows, cols))).to(dtype)


def _tolerance(x, dtype, math, groups=None, **kw):
    x = _np(x)
    off = R.newton_schulz_fp16(x, groups=groups, **kw)
    ref = R.orthogonalize(x, **kw)
    off = off.T if x.shape[0] > x.shape[1] else off
    e = np.linalg.norm(off - ref) / np.linalg.norm(ref)
    return ref, (1.5 * e if math == HALF else e * 2.0 ** -8) + U[dtype] + 2.0 ** -22


def _check(got, ref, tol):
    off = np.linalg.norm(_np(got) - ref) / np.linalg.norm(ref)
    assert off <= tol, (off, tol)


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    assert K.operator_status() == (0, 0)


# a lone element, vectors; up to 128 on one side by one block and by clusters of two, four and eight,
# and too long for them; one tile and its borders, several tiles of either orientation
SIZES = [(1, 1), (1, 7), (9, 1), (5, 3), (16, 16), (40, 64), (64, 65), (33, 100), (100, 33), (128, 128),
         (128, 512), (129, 512), (128, 513), (77, 1000), (1024, 100), (128, 1025), (2047, 65), (17, 2049),
         (128, 4096), (4096, 9), (4097, 40), (130, 500), (256, 256), (257, 300), (300, 257), (513, 1000), (1000, 513), (520, 2100), (2100, 260)]


@pytest.mark.parametrize("dtype,math", [(BF16, HALF), (F32, FULL), (F32, HALF), (BF16, FULL)])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_orthogonalize(dtype, math, rows, cols):
    x = _gradient(rows + cols, rows, cols, dtype)
    keep = x.clone()
    ref, tol = _tolerance(x, dtype, math)
    got = K.orthogonalize(x, math=math)
    assert got.dtype is dtype and torch.equal(x, keep)
    _check(got, ref, tol)
    assert torch.equal(got, K.orthogonalize(x, math=math))   # the same bits


@pytest.mark.parametrize("dtype,math", [(BF16, HALF), (F32, FULL), (F32, HALF), (BF16, FULL)])
@pytest.mark.parametrize("rows,cols", [(1024, 1600), (2100, 1030)])
def test_long_matrices_take_steps_in_groups(dtype, math, rows, cols):
    x = _gradient(rows + cols, rows, cols, dtype)
    ref, tol = _tolerance(x, dtype, math, groups=(3, 2))
    _check(K.orthogonalize(x, math=math), ref, tol)
    if math == HALF and dtype is BF16:
        # a first step that lifts small values more (L's rounding by 4.2^2 11.9 > 150): a group of two
        co = [(4.2, -10.5, 7.35)] + [(3.4445, -4.7750, 2.0315)] * 2
        want = R.orthogonalize(_np(x), 3, co)
        # the roundings are those of the default's three; the first step lifts them 4.2 / 3.4445 times more
        _, tol = _tolerance(x, dtype, math, groups=(2, 1), steps=3)
        _check(K.orthogonalize(x, steps=3, coefficients=co), want, 4.2 / 3.4445 * tol)
        # these would take singular values to 2.06, then to 45, then past every bound
        with pytest.raises(K.KfacError, match="INVALID_ARG"):
            K.orthogonalize(x, steps=3, coefficients=[(8.0, -20.0, 14.0)] + co[1:])
        # one step alone, and steps that are not a whole number of groups
        for steps, groups in ((1, (1,)), (4, (3, 1)), (7, (3, 3, 1))):
            ref, tol = _tolerance(x, dtype, math, groups=groups, steps=steps)
            _check(K.orthogonalize(x, steps=steps), ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_matrices_at_once(dtype):
    """More than one launch takes, of all kinds, each as by itself; defaults by type."""
    rng = np.random.default_rng(0)
    draws = [tuple(rng.integers(1, 400, 2)) for _ in range(60)]
    empty = [(0, 5), (4, 0)]
    small = [s for s in draws if min(s) <= 128] + [(600, 90), (90, 700)] + empty
    large = [s for s in draws if min(s) > 128] + [(1024, 1536)] + empty
    for shapes in (small, large, small + large):
        xs = [_gradient(i, *s, dtype) for i, s in enumerate(shapes)]
        ws = K.orthogonalize_workspace(xs)
        ws.fill_(255)     # whatever an earlier call left there: NaNs
        got = K.orthogonalize(xs, workspace=ws)
        for x, y in zip(xs, got):
            assert y.shape == x.shape
            if x.numel():
                assert torch.equal(y, K.orthogonalize(x))
    # a few small ones beside a large one: the large one's launches take them
    xs = [_gradient(i, *s, dtype) for i, s in enumerate([(300, 200), (10, 700), (33, 20), (600, 128), (0, 3)])]
    got = K.orthogonalize(xs)
    again = K.orthogonalize(xs)
    assert torch.equal(got[0], K.orthogonalize(xs[0]))
    for x, y, z in list(zip(xs, got, again))[:4]:
        ref, tol = _tolerance(x, dtype, HALF if dtype is BF16 else FULL)
        _check(y, ref, tol)
        assert torch.equal(y, z)
    stacked = torch.stack([_gradient(i, 70, 130, dtype) for i in range(3)])
    got = K.orthogonalize(stacked)
    assert got.shape == stacked.shape
    for i in range(3):
        assert torch.equal(got[i], K.orthogonalize(stacked[i]))


def test_steps_and_coefficients():
    x = _gradient(1, 60, 90, BF16)
    for kw in (dict(steps=1), dict(steps=2), dict(steps=8, coefficients=(1.5, -0.5, 0.0)),
               dict(steps=3, coefficients=(2.0, -1.5, 0.5)), dict(steps=5, eps=1.0)):
        ref, tol = _tolerance(x, BF16, HALF, **kw)
        _check(K.orthogonalize(x, **kw), ref, tol)
    per_step = [(3.4445, -4.7750, 2.0315)] * 3 + [(1.5, -0.5, 0.0)] * 2
    want = R.orthogonalize(_np(x), 5, per_step)
    _, tol = _tolerance(x, BF16, HALF)
    _check(K.orthogonalize(x, coefficients=per_step), want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_in_place(dtype):
    wide = _gradient(1, 300, 500, dtype)
    for rows in (300, 60):
        x = wide[:rows, 3:180]               # rows of odd alignment
        want = K.orthogonalize(x.contiguous())
        out = torch.full((rows + 1, 200), 7.0, device="cuda", dtype=dtype)
        assert torch.equal(K.orthogonalize(x, out=out[:rows, 5:182]), want)
        assert (out[:, :5] == 7).all() and (out[:, 182:] == 7).all() and (out[rows] == 7).all()
        rest = wide[:, 180:].clone()
        K.orthogonalize(x, out=x)
        assert torch.equal(x, want) and torch.equal(wide[:, 180:], rest)
        wide = _gradient(2, 300, 500, dtype)


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-12, 1e12, 1e30])
@pytest.mark.parametrize("rows,cols", [(65, 40), (50, 700), (140, 200)])
def test_scale_of_the_matrix_does_not_matter(size, rows, cols):
    x = _gradient(1, rows, cols, size=1.0)
    x = (x.double() * size).float()
    ref = R.orthogonalize(_np(x), eps=0.0)    # (1e-42: denormals, the few bits that they have)
    _, tol = _tolerance(x, F32, FULL, eps=0.0)
    _check(K.orthogonalize(x, eps=0.0), ref, tol)


@pytest.mark.parametrize("math", [FULL, HALF])
def test_zeros_and_what_is_not_finite_stay_where_they_are(math):
    for rows, cols in ((150, 70), (150, 170), (60, 1000)):
        xs = [_gradient(i, rows, cols) for i in range(5)]
        xs[1].zero_()
        xs[2][rows - 1, cols - 1] = float("nan")
        xs[3][0, 1] = float("inf")
        got = K.orthogonalize(xs, math=math)
        assert (got[1] == 0).all() and torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
        for i in (0, 4):
            assert torch.equal(got[i], K.orthogonalize(xs[i], math=math))
        assert (K.orthogonalize(xs[1], eps=0.0, math=math) == 0).all()


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype,math", [(F32, None), (F32, HALF), (BF16, None)])
def test_step(dtype, math, nesterov):
    """Two steps of several matrices; rows of any alignment."""
    shapes = [(64, 64), (10, 300), (300, 33), (257, 256), (90, 1100), (700, 120)]
    kw = dict(lr=0.05, momentum=0.9, weight_decay=0.1, nesterov=nesterov, update_scale=0.7)
    gs = [[_gradient(10 * k + i, *s, dtype) for i, s in enumerate(shapes)] for k in range(2)]
    ms = [_gradient(50 + i, *s) for i, s in enumerate(shapes)]
    ws = [torch.randn(s[0], s[1] + 3, device="cuda")[:, 1:-2] * s[1] ** -0.5 for s in shapes]
    rm, rw = [_np(m) for m in ms], [_np(w) for w in ws]
    sizes = [np.abs(m) for m in rm]
    work = K.orthogonalize_workspace(gs[0], math=math)
    use = math if math is not None else (HALF if dtype is BF16 else FULL)
    for k in range(2):
        K.orthogonal_step(gs[k], ms, ws, math=math, workspace=work, **kw)
        for i, s in enumerate(shapes):
            before = rw[i]
            rm[i], rw[i] = R.orthogonal_step(_np(gs[k][i]), rm[i], rw[i], **kw)
            # the momentum: mu's rounding and two of the terms, whose sum may be far smaller than they
            # are; the error of the step before it comes in times mu, and is measured by the terms
            # there, not by what they left: e' <= mu e + 3 f (mu |m| + |g|) with size' = mu size + |g|
            # gives e <= 3 f (k + 1) size
            sizes[i] = 0.9 * sizes[i] + np.abs(_np(gs[k][i]))
            assert (np.abs(_np(ms[i]) - rm[i]) <= 8 * 2.0 ** -24 * sizes[i]).all()
            u = torch.from_numpy(_np(gs[k][i]) + 0.9 * rm[i] if nesterov else rm[i]).cuda()
            _, tol = _tolerance(u, F32, use)
            # the direction's error, at most twice over with the step before it, and the weights' own
            move = 0.05 * 0.7 * np.sqrt(max(1, s[0] / s[1]) * min(s)) * 1.21
            off = np.linalg.norm(_np(ws[i]) - rw[i])
            assert off <= 2 * tol * move + 8 * 2.0 ** -24 * np.linalg.norm(before)


def test_streams_and_graphs():
    """On another stream; two captured calls with workspaces of their own, replayed in turn."""
    xs = [_gradient(i, 200, 300, BF16) for i in range(2)]
    small = _gradient(5, 40, 900, BF16)
    done = torch.empty_like(small)
    once = K.orthogonalize(small)
    want = [K.orthogonalize(x) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = K.orthogonalize(xs[0], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])
    graphs = []
    for x in xs:
        out = torch.empty_like(x)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            K.orthogonalize(x, out=out)
            K.orthogonalize(small, out=done)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out.fill_(5)
            g.replay()
    for (_, out), w in zip(graphs, want):
        assert torch.equal(out, w)
    assert torch.equal(done, once)
    xs[0].copy_(xs[1])       # a replay reads the present values
    graphs[0][0].replay()
    assert torch.equal(graphs[0][1], want[1])


def test_python_refusals():
    x = torch.zeros(4, 6, device="cuda")
    with pytest.raises(ValueError, match="matrices"):
        K.orthogonalize([x, x], out=[x])
    with pytest.raises(ValueError, match="holds"):
        K.orthogonal_step([x], [x.bfloat16()], [x], lr=0.1)
    with pytest.raises(ValueError, match="holds"):
        K.orthogonalize([x, x.bfloat16()])
    with pytest.raises(ValueError, match="contiguous"):
        K.orthogonalize(x.t())
    with pytest.raises(ValueError, match="2-D|rows, columns"):
        K.orthogonalize(x[0])
    with pytest.raises(K.KfacError, match="INVALID_ARG"):
        K.orthogonalize([x, x + 1], out=[x, x])
    assert K.orthogonalize([]) == [] and K.orthogonalize([x[:0], x[:, :0]])[0].shape == (0, 6)
    with pytest.raises(K.KfacError, match="WORKSPACE"):
        K.orthogonalize(torch.zeros(150, 200, device="cuda"),
                        workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_sides_that_no_int_holds_are_refused():
    """2^32 + 1 rows (of one stored row) are not taken for one row."""
    x = torch.ones(8, device="cuda").as_strided((2**32 + 1, 8), (0, 1))
    with pytest.raises(K.KfacError, match="UNSUPPORTED"):
        K.orthogonalize(x, out=x)
    with pytest.raises(K.KfacError, match="UNSUPPORTED"):
        K.orthogonalize_workspace(x)
    with pytest.raises(K.KfacError, match="UNSUPPORTED"):
        K.orthogonal_step(x, x, x, lr=0.1)


def test_matrices_from_an_iterator():
    xs = [_gradient(i, 30 + i, 40) for i in range(3)]
    want = K.orthogonalize(xs)
    got = K.orthogonalize(x for x in xs)
    assert len(got) == 3 and all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(x) for x in xs]
    got = K.orthogonalize(iter(xs), out=iter(out))
    assert len(got) == 3 and all(a is b and torch.equal(a, c) for a, b, c in zip(got, out, want))
