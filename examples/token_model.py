"""Train a small token model with a step for every kind of parameter:

    h = embedding(ids);  per layer: h = h + W2 relu(W1 norm(h));  logits = H norm(h)

The head's weights H are stepped by K-FAC (Kronecker factors), the matrices W1 and W2 along their
orthogonalised momentum (K.orthogonal_step), the table and the norms' gains by the diagonal step: their
factors are what the embedding's and the norms' backward passes give (the tokens' frequencies, the
mean squares of the gains' gradients).  The matrix products are torch's; the embedding, the norms with
the residual's addition and the steps are the package's.

    python examples/token_model.py [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import second_order_optimizer_gb300 as K  # noqa: E402


class Model:
    """fp32 parameters, bf16 activations."""

    def __init__(self, vocabulary, width, inner, layers, max_tokens, seed=0, lr=2e-2):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.vocabulary, self.width, self.layers, self.lr = vocabulary, width, layers, lr
        self.table = draw(vocabulary, width) * width ** -0.5
        self.scale = width ** 0.5
        self.w = [draw(*s) * s[1] ** -0.5 for _ in range(layers) for s in ((inner, width), (width, inner))]
        self.momenta = [torch.zeros_like(w) for w in self.w]
        self.gains = [torch.ones(width, device="cuda") for _ in range(layers + 1)]
        self.head = draw(vocabulary, width) * width ** -0.5
        # layers of the handle: the head, the table, the gains
        self.kfac = K.Kfac([(K.KFAC_KRON, vocabulary, width, 0, K.KFAC_BF16),
                            (K.KFAC_DIAG, vocabulary, width, 0, K.KFAC_BF16)] +
                           [(K.KFAC_DIAG, width, 1, 0, K.KFAC_F32) for _ in self.gains],
                           max_rows=max_tokens, lr=lr, damping=1e-3, momentum=0.9, weight_decay=0.0)
        self.one = torch.ones(1, device="cuda")
        self.ortho = K.orthogonalize_workspace(self.w)
        self.count = 0

    def forward(self, ids):
        """Logits (bf16) of the tokens; keeps what the backward pass reads."""
        h = K.embedding(ids, self.table.bfloat16(), scale=self.scale)
        saved, add = [], None
        w = [t.bfloat16() for t in self.w]
        for i in range(self.layers):
            n, s, rstd = K.rms_norm(h, self.gains[i], residual=add)
            h = h if s is None else s                      # the stream, the last layer's output added
            z = torch.relu(n @ w[2 * i].t())
            saved.append((n, h, rstd, z))
            add = z @ w[2 * i + 1].t()
        n, h, rstd = K.rms_norm(h, self.gains[-1], residual=add)
        self.saved = (ids, saved, (n, h, rstd), w)
        return n @ self.head.bfloat16().t()

    def backward(self, dlogits):
        """Gradients of every parameter for those of the logits (bf16): a dict."""
        ids, saved, (n, h, rstd), w = self.saved
        g = {"head_in": n, "head_out": dlogits, "w": [None] * len(w), "gains": [None] * (self.layers + 1)}
        dh, *g["gains"][self.layers:] = self._norm_back(dlogits @ self.head.bfloat16(), h, self.layers, rstd)
        for i in reversed(range(self.layers)):
            n, h, rstd, z = saved[i]
            # dh is the gradient of the stream and of what the layer added to it
            g["w"][2 * i + 1] = dh.t().float() @ z.float()
            dz = (dh @ w[2 * i + 1]) * (z > 0)
            g["w"][2 * i] = dz.t().float() @ n.float()
            dh, g["gains"][i] = self._norm_back(dz @ w[2 * i], h, i, rstd, dh)
        g["frequency"] = torch.empty(self.vocabulary, device="cuda")
        g["table"] = K.embedding_backward(ids, dh, self.vocabulary, scale=self.scale,
                                          frequency=g["frequency"])
        g["embedded"] = dh
        return g

    def _norm_back(self, dn, h, i, rstd, dresidual=None):
        dx, dgain, square = K.rms_norm_backward(dn, h, self.gains[i], rstd, dresidual=dresidual, square=True)
        return dx, (dgain, square)

    def step(self, ids, targets, refresh_every=5):
        """One step on the mean cross entropy; returns the loss (a device scalar)."""
        logits = self.forward(ids)
        rows = ids.numel()
        p = torch.softmax(logits.float(), dim=-1)
        loss = -torch.log(p.gather(1, targets[:, None]) + 1e-30).mean()
        p.scatter_add_(1, targets[:, None], torch.full_like(targets[:, None], -1.0, dtype=p.dtype))
        g = self.backward(p.bfloat16())                    # of the sum over the tokens
        # the head: Kronecker factors from its input and output gradients
        self.kfac.update_factors(0, g["head_in"], g["head_out"])
        if self.count % refresh_every == 0:
            self.kfac.invert(0)
        dhead = (g["head_out"].t().float() @ g["head_in"].float()) / rows
        self.kfac.precondition(0, dhead, None, None, None, self.head, None)
        # the matrices: their scale does not matter to the direction
        K.orthogonal_step(g["w"], self.momenta, self.w, lr=self.lr, workspace=self.ortho)
        # the table: A of the one-hot inputs is the tokens' frequencies, G the mean squares of dh
        e = g["embedded"].float()
        squares = (e * e).mean(dim=0) * self.scale ** 2
        self.kfac.diag_step(1, g["frequency"], squares, g["table"] / rows, None, self.table, None)
        for i, (dgain, square) in enumerate(g["gains"]):
            self.kfac.diag_step(2 + i, square, self.one, dgain / rows, None, self.gains[i], None)
        self.count += 1
        return loss


def train(steps=40, tokens=512, vocabulary=97, width=128, inner=256, layers=2, seed=0):
    """Learn a fixed map from token to next token; returns the losses."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    follows = torch.randperm(vocabulary, generator=gen, device="cuda")
    model = Model(vocabulary, width, inner, layers, tokens, seed)
    losses = []
    for _ in range(steps):
        ids = (vocabulary * torch.rand(tokens, generator=gen, device="cuda") ** 2).long()
        losses.append(model.step(ids, follows[ids]))
    code, layer, info = model.kfac.get_status()
    assert code == 0, (code, layer, info)
    assert K.operator_status()[0] == 0
    return [float(l) for l in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    ls = train(a.steps)
    for i, l in enumerate(ls):
        if i % max(1, len(ls) // 10) == 0 or i == len(ls) - 1:
            print(f"step {i:4d}  loss {l:.5f}")
