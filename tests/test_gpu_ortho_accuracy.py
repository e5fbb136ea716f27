"""GPU accuracy of the orthogonalised updates on matrices other than full-rank ones of an ordinary norm.

Tolerances in norm, fixed before the first run, by the roundings of the reference's own iteration as in
test_gpu_ortho.py: half arithmetic 1.5 e, full arithmetic e 2^-8, each and the result's own rounding.  e
is of the iteration that stores the products on the small side by their upper half on both sides, as the
kernels do: where steps are taken in groups there, roundings that are equal in pairs add up to more than
independent ones do (1030 x 1600: 2.4e-3 for 1.8e-3 at an ordinary norm, 3.1e-3 for 1.9e-3 at |x| = eps).
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
FORMS = [(F32, FULL), (F32, HALF), (BF16, HALF)]


def _randn(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def _gradient(seed, rows, cols):
    """A few strong directions and noise."""
    r = max(1, min(rows, cols) // 8)
    strong = np.logspace(0, -1, r)
    return (_randn(seed, rows, r) * strong) @ _randn(seed + 1, r, cols) / r ** 0.5 + 0.2 * _randn(seed + 2, rows, cols)


def _off(x, dtype, math, groups=None, **kw):
    """(distance from float64, tolerance)"""
    t = torch.from_numpy(x).to("cuda", dtype)
    x = t.double().cpu().numpy()
    ref = R.orthogonalize(x, **kw)
    e = R.newton_schulz_fp16(x, groups=groups, mirror=True, **kw)
    e = np.linalg.norm((e.T if x.shape[0] > x.shape[1] else e) - ref) / np.linalg.norm(ref)
    got = K.orthogonalize(t, math=math, **kw).double().cpu().numpy()
    assert K.operator_status() == (0, 0)
    return (np.linalg.norm(got - ref) / np.linalg.norm(ref),
            (1.5 * e if math == HALF else e * 2.0 ** -8) + U[dtype] + 2.0 ** -22)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("norm", [1e-6, 1e-7, 1e-9, 1e-11, 1e-13, 1e-15, 1e-20])
def test_matrices_far_below_eps(norm, dtype, math):
    """Norms down to 1e-13 of eps: X is as small from its first step to its last, and as exact as any."""
    for rows, cols, groups in ((65, 40, None), (50, 700, None), (140, 200, None), (1030, 1600, (3, 2))):
        x = _gradient(rows, rows, cols)
        off, tol = _off(x * (norm / np.linalg.norm(x)), dtype, math, groups)
        assert off <= tol, (rows, cols, off, tol)
    # other polynomials, other eps
    for rows, cols in ((90, 130), (140, 150)):
        x = _gradient(3, rows, cols)
        x *= norm / 30 / np.linalg.norm(x)
        for kw in (dict(steps=12, coefficients=(1.5, -0.5, 0.0)), dict(steps=1),
                   dict(steps=3, coefficients=(0.5, 0.0, 0.0)), dict(eps=1.0), dict(eps=1e6)):
            off, tol = _off(x, dtype, math, **kw)
            assert off <= tol, (rows, cols, kw, off, tol)


def test_eps_beyond_fp32():
    for rows, cols in ((150, 200), (60, 90)):
        x = torch.from_numpy(_gradient(1, rows, cols)).to("cuda", F32)
        assert (K.orthogonalize(x, eps=1e300) == 0).all()
        x[0, 0] = float("inf")
        assert torch.isnan(K.orthogonalize(x, eps=1e300)).all()


def _low_rank(rows, cols, rank):
    return _randn(rank, rows, rank) @ _randn(rank + 1, rank, cols)


def _falling(rows, cols, least):
    """Singular values from 1 to `least`, evenly in their logarithm."""
    s = min(rows, cols)
    u, v = np.linalg.qr(_randn(5, rows, s))[0], np.linalg.qr(_randn(6, cols, s))[0]
    return (u * np.logspace(0, np.log10(least), s)) @ v.T


SPECTRA = [(256, 512, None), (60, 1000, None), (700, 120, None), (1030, 1600, (3, 2))]


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols,groups", SPECTRA)
def test_low_rank(rows, cols, groups, dtype, math):
    """Gradients of fewer tokens than channels: the steps lift what rounding leaves in the empty
    directions, by up to 3.4445^5."""
    for rank in (1, 4, min(rows, cols) // 8):
        off, tol = _off(_low_rank(rows, cols, rank), dtype, math, groups)
        assert off <= tol, (rank, off, tol)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols,groups", SPECTRA)
def test_falling_spectra(rows, cols, groups, dtype, math):
    for least in (1e-2, 1e-4, 1e-6):
        off, tol = _off(_falling(rows, cols, least), dtype, math, groups)
        assert off <= tol, (least, off, tol)
