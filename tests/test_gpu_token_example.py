"""The example that steps every kind of parameter: that it runs, and its gradients against float64."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_model as E  # noqa: E402


def test_example_runs():
    losses = E.train(steps=8)
    assert len(losses) == 8 and np.isfinite(losses).all()


@pytest.mark.parametrize("layers", [1, 3])
def test_example_gradients_against_float64(layers):
    """Every parameter's gradient for given gradients of the logits, against torch's differentiation of
    the same model in float64 (on the parameters that its products see: rounded to bf16).

    In norm: each activation and gradient between the parameters is rounded to bf16 (u = 2^-8) where it
    is stored, at most four of them per layer on the way there and four back, besides the logits'
    gradient and the table's rows: 8 layers + 6 roundings, each at most u of what it rounds, and a
    relu's border is crossed by values within u of it (the same size)."""
    v, width, inner, t = 61, 64, 96, 300
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    m = E.Model(v, width, inner, layers, t, seed=1)
    ids = torch.randint(0, v - 5, (t,), generator=gen, device="cuda")
    dlogits = torch.randn(t, v, generator=gen, device="cuda").bfloat16()
    m.forward(ids)
    g = m.backward(dlogits)

    leaf = lambda x: x.bfloat16().double().requires_grad_(True)
    table, w, head = leaf(m.table), [leaf(x) for x in m.w], m.head.bfloat16().double()
    gains = [x.double().requires_grad_(True) for x in m.gains]
    norm = lambda x, gain: x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gain
    h = table[ids] * m.scale
    for i in range(layers):
        h = h + torch.relu(norm(h, gains[i]) @ w[2 * i].t()) @ w[2 * i + 1].t()
    (norm(h, gains[-1]) @ head.t()).backward(dlogits.double())
    tol = (8 * layers + 6) * 2.0 ** -8
    pairs = [(g["table"], table.grad)] + list(zip(g["w"], [x.grad for x in w]))
    pairs += [(a[0], b.grad) for a, b in zip(g["gains"], gains)]
    for got, ref in pairs:
        assert got.shape == ref.shape
        assert float((got.double() - ref).norm() / ref.norm()) <= tol
    freq = torch.bincount(ids, minlength=v).double() / t
    assert torch.allclose(g["frequency"].double(), freq, rtol=2.0 ** -22, atol=0)
    assert (g["table"][v - 5:] == 0).all()
