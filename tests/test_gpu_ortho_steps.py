"""GPU parity of kfac_orthogonal_step in each of the kernels that write weights: the small matrices' own,
CTA pairs on 256 x 256 tiles, single steps and steps taken in groups, both arithmetics.

Tolerances as in test_gpu_ortho_accuracy.py, fixed before the first run; the weights' own rounding and the
momentum's beside it.
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
FORMS = [(F32, FULL), (F32, HALF), (BF16, HALF), (BF16, FULL)]
LR, MU, DECAY, SCALE = 0.05, 0.9, 0.1, 0.7


def _np(t):
    return t.detach().double().cpu().numpy()


def _gradient(seed, rows, cols, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    r = max(1, min(rows, cols) // 8)
    strong = torch.logspace(0, -1, r, device="cuda")
    return (1e-4 * ((randn(rows, r) * strong) @ randn(r, cols) / r ** 0.5 + 0.2 * randn(rows, cols))).to(dtype)


def _run(shapes, dtype, math, nesterov, groups=None, steps=2):
    gs = [[_gradient(10 * k + i, *s, dtype) for i, s in enumerate(shapes)] for k in range(steps)]
    ms = [_gradient(50 + i, *s, F32) for i, s in enumerate(shapes)]
    # rows of any alignment, with something beside them that stays
    wide = [torch.randn(s[0], s[1] + 3, device="cuda") * s[1] ** -0.5 for s in shapes]
    beside = [w.clone() for w in wide]
    ws = [w[:, 1:-2] for w in wide]
    rm, rw = [_np(m) for m in ms], [_np(w) for w in ws]
    size = [np.abs(m) for m in rm]
    off = [0.0] * len(shapes)
    work = K.orthogonalize_workspace(gs[0], math=math)
    for k in range(steps):
        K.orthogonal_step(gs[k], ms, ws, lr=LR, momentum=MU, weight_decay=DECAY, nesterov=nesterov,
                          update_scale=SCALE, math=math, workspace=work)
        assert K.operator_status() == (0, 0)
        for i, s in enumerate(shapes):
            g, before = _np(gs[k][i]), rw[i]
            rm[i], rw[i] = R.orthogonal_step(g, rm[i], before, LR, MU, DECAY, nesterov, SCALE)
            # momentum: mu's rounding and one fused product and sum: 2 2^-24 of the terms each step, and mu
            # times what was there; within 4 2^-24 of the sum of the terms' sizes
            size[i] = MU * size[i] + np.abs(g)
            assert (np.abs(_np(ms[i]) - rm[i]) <= 4 * 2.0 ** -24 * size[i]).all()
            u = (g + MU * rm[i] if nesterov else rm[i])
            u = u.astype(np.float32).astype(np.float64)
            ref = R.orthogonalize(u)
            e = R.newton_schulz_fp16(u, groups=groups, mirror=True)
            e = np.linalg.norm((e.T if s[0] > s[1] else e) - ref)
            tol = 1.5 * e if math == HALF else e * 2.0 ** -8
            # 2^-21: u's own rounding, of another momentum than the reference's, lifted by at most 3.4445^5
            # where the direction hardly has it: 4 2^-24 485 of a part of u of 2^-10 its norm
            tol += 2.0 ** -21 * np.linalg.norm(ref) * (4 if k else 1)
            rate = LR * SCALE * np.sqrt(max(1, s[0] / s[1]))
            off[i] = off[i] * (1 - LR * DECAY) + rate * tol + 4 * 2.0 ** -24 * np.linalg.norm(before)
            got = np.linalg.norm(_np(ws[i]) - rw[i])
            assert got <= off[i], (s, k, got, off[i])
            # and the step is one: it moved the weights by what the reference's did
            assert np.linalg.norm(rw[i] - before) > 20 * off[i]
    for a, b in zip(wide, beside):
        assert torch.equal(a[:, :1], b[:, :1]) and torch.equal(a[:, -2:], b[:, -2:])


# one block; clusters of two, four and eight, wide and tall; vectors
SMALL = [(64, 64), (1, 9), (100, 33), (10, 300), (128, 512), (90, 1100), (700, 120), (128, 1400), (1500, 40)]


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("dtype,math", FORMS)
def test_small_matrices_by_themselves(dtype, math, nesterov):
    _run(SMALL, dtype, math, nesterov)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", [(2000, 130), (4, 4090)])
def test_one_matrix(rows, cols, dtype, math):
    _run([(rows, cols)], dtype, math, True)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols,groups", [(1700, 1800, None), (1040, 2200, (3, 2)), (2200, 1040, (3, 2))])
def test_pairs(rows, cols, groups, dtype, math):
    """More 256 x 256 tiles than a quarter of the SMs, at ragged sizes."""
    _run([(rows, cols)], dtype, math, rows != 1700, groups, steps=1)


@pytest.mark.parametrize("dtype,math", FORMS[:1] + FORMS[2:3])
def test_small_ones_beside_a_large_one_on_pairs(dtype, math):
    _run([(1700, 1800), (20, 300), (120, 64)], dtype, math, True, steps=1)
