"""The example that runs the block operators together with the optimizer step: its gradients
against float64, and that it trains."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import cross_attention_block as E  # noqa: E402
from oracle import block_oracle as B  # noqa: E402


def test_example_trains():
    losses = E.train(steps=30)
    assert np.isfinite(losses).all()
    # dropout at p = 0.1 leaves a floor; the fit gets rid of most of the rest
    assert np.mean(losses[-5:]) < 0.6 * losses[0]


def test_example_gradients_against_float64():
    """dL/dy -> the projections' output gradients, through dropout, attention and the rotations,
    with the block's own bf16 intermediates promoted to float64."""
    b, n, m, width, heads, kv = 2, 21, 45, 128, 4, 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    blk = E.Block(width, heads, kv, b, n, m, seed=1, p=0.25)
    x, e, dy = draw(b, n, width), draw(b, m, width), draw(b, n, width)
    kv_len = torch.tensor([0, 37], device="cuda", dtype=torch.int32)
    blk.forward(x, e, kv_len)
    _, _, _, q, k, v, a, lse, w = blk.saved
    inputs, grads = blk.backward(dy)
    f = lambda t: t.double().cpu().numpy()
    dh = B.dropout(f(dy), 0.25, 1, 0)
    dh16 = torch.from_numpy(dh).bfloat16().cuda()   # the block's own rounding
    assert np.array_equal(f(grads[E.O]).reshape(dh.shape), f(dh16))
    da = f((dh16 @ w[E.O]).view_as(a))
    ok = B.permitted(b, m, [0, 37])
    dq, dk, dv = B.cross_attention_backward(da, f(q), f(k), f(v), ok)
    table = f(blk.table)
    pos = lambda t: np.broadcast_to(np.arange(t.shape[1]), t.shape[:2])
    dq, dk = B.rope(dq, table, pos(dq), inverse=True), B.rope(dk, table, pos(dk), inverse=True)
    for got, ref in ((grads[E.Q], dq), (grads[E.KEY], dk), (grads[E.V], dv)):
        ref = ref.reshape(f(got).shape)
        # operands, delta and results rounded to bf16 (u = 2^-8): at most 4 u in norm
        assert np.linalg.norm(f(got) - ref) <= 4 * 2.0 ** -8 * np.linalg.norm(ref)
    assert (f(grads[E.V]).reshape(b, -1)[0] == 0).all()   # the sequence without encoder states
