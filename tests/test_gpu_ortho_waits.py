"""Orthogonalised updates whose waits give up: the self-test takes one wait of a product launch for one
that ran out.  The call ends, says so once, and what runs behind it is not disturbed."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import second_order_optimizer_gb300 as K  # noqa: E402
from second_order_optimizer_gb300._lib import LIB  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
TIMEOUT = 5
FORMS = [(BF16, K.KFAC_ORTHO_HALF), (F32, K.KFAC_ORTHO_FULL)]
# single CTAs on 128 x 128 tiles; CTA pairs on 256 x 256 ones
SIZES = [(300, 500), (2304, 2400)]


def _matrix(rows, cols, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda").to(dtype)


def _selftest(launch):
    assert LIB.kfac_selftest_orthogonal(launch) == 0


LAUNCHES = 15   # of five single steps: X X^T, M, M X each


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_last_product(rows, cols, dtype, math):
    """The rows of the warp that gave up are NaN; then the same call on the same workspace is right."""
    x = _matrix(rows, cols, dtype)
    work = K.orthogonalize_workspace(x, math=math)
    want = K.orthogonalize(x, math=math, workspace=work)
    for _ in range(3):
        _selftest(LAUNCHES - 1)
        got = K.orthogonalize(x, math=math, workspace=work)
        code, info = K.operator_status()
        assert code == TIMEOUT and info in (44, 45)
        assert torch.isnan(got[:32, :32]).all() and not torch.isnan(want).any()
        kept = ~torch.isnan(got)
        assert torch.equal(got[kept], want[kept])
        assert K.operator_status() == (0, 0)
        assert torch.equal(K.orthogonalize(x, math=math, workspace=work), want)
        assert K.operator_status() == (0, 0)


def test_selftest_is_of_one_call():
    assert LIB.kfac_selftest_orthogonal(-2) == 1
    x = _matrix(300, 500, BF16)
    want = K.orthogonalize(x)
    _selftest(3)
    _selftest(-1)
    assert torch.equal(K.orthogonalize(x), want) and K.operator_status() == (0, 0)
    _selftest(LAUNCHES)   # none of this number
    assert torch.equal(K.orthogonalize(x), want)
    assert torch.equal(K.orthogonalize(x), want) and K.operator_status() == (0, 0)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("launch", [0, 1, 2, 13])
def test_product_on_the_way(rows, cols, dtype, math, launch):
    """One warp of four that store together gives up; the others, whose products are done, do not wait
    for it."""
    x = _matrix(rows, cols, dtype)
    work = K.orthogonalize_workspace(x, math=math)
    want = K.orthogonalize(x, math=math, workspace=work)
    for _ in range(3):
        _selftest(launch)
        K.orthogonalize(x, math=math, workspace=work)
        code, info = K.operator_status()
        assert code == TIMEOUT and info in (44, 45) and K.operator_status() == (0, 0)
        assert torch.equal(K.orthogonalize(x, math=math, workspace=work), want)
        assert K.operator_status() == (0, 0)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("launch", [0, 1, 2, 7, 13])
def test_a_lost_product_reaches_the_result(rows, cols, dtype, math, launch):
    """All of the matrix's direction is NaN, whatever earlier calls left in the workspace; the matrices
    beside it are right."""
    xs = [_matrix(rows, cols, dtype), _matrix(200, 300, dtype), _matrix(260, 140, dtype)]
    work = K.orthogonalize_workspace(xs, math=math)
    want = K.orthogonalize(xs, math=math, workspace=work)
    _selftest(launch)
    got = K.orthogonalize(xs, math=math, workspace=work)
    assert K.operator_status()[0] == TIMEOUT
    # (with 128 x 128 tiles the block that gave up has none of the others' tiles behind its first)
    assert torch.isnan(got[0]).all()
    for x, y in zip(got[1:], want[1:]):
        assert torch.equal(x, y) or torch.isnan(x).all()
    assert sum(bool(torch.isnan(x).any()) for x in got) < 3
    for x, y in zip(K.orthogonalize(xs, math=math, workspace=work), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("launch", [0, 7, 13, 14])
def test_weights_keep_their_values(rows, cols, dtype, math, launch):
    g, m0, w0 = _matrix(rows, cols, dtype), _matrix(rows, cols, F32, 1), _matrix(rows, cols, F32, 2)
    work = K.orthogonalize_workspace(g, math=math)
    m, w = m0.clone(), w0.clone()
    K.orthogonal_step(g, m, w, lr=0.1, weight_decay=0.1, math=math, workspace=work)
    stepped, moved = m.clone(), w.clone()
    m.copy_(m0)
    w.copy_(w0)
    _selftest(launch)
    K.orthogonal_step(g, m, w, lr=0.1, weight_decay=0.1, math=math, workspace=work)
    assert K.operator_status()[0] == TIMEOUT
    assert torch.equal(m, stepped)
    if launch < LAUNCHES - 1:
        assert torch.equal(w, w0)
    else:   # of the last product what gave up keeps its weights, the rest has moved
        assert torch.equal(w[:32, :32], w0[:32, :32]) and ((w == w0) | (w == moved)).all()


# one block; clusters of two to eight; both orientations
SMALL = [(100, 90), (60, 1000), (1000, 128), (128, 1400), (1500, 30)]


@pytest.mark.parametrize("dtype,math", FORMS)
@pytest.mark.parametrize("rows,cols", SMALL)
@pytest.mark.parametrize("step", [0, 2, 4])
def test_small_matrices_give_up_as_a_cluster(rows, cols, dtype, math, step):
    x = _matrix(rows, cols, dtype)
    want = K.orthogonalize(x, math=math)
    _selftest(step)
    got = K.orthogonalize(x, math=math)
    code, info = K.operator_status()
    assert (code, info) == (TIMEOUT, 46)
    assert torch.isnan(got).all()
    assert torch.equal(K.orthogonalize(x, math=math), want)
    m, w0 = _matrix(rows, cols, F32, 1), _matrix(rows, cols, F32, 2)
    w = w0.clone()
    _selftest(step)
    K.orthogonal_step(x, m, w, lr=0.1, weight_decay=0.1, math=math)
    assert K.operator_status()[0] == TIMEOUT and torch.equal(w, w0)
    K.orthogonal_step(x, m, w, lr=0.1, weight_decay=0.1, math=math)
    assert K.operator_status() == (0, 0) and not torch.isnan(w).any() and (w != w0).any()
