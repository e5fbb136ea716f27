"""Train one decoder block that reads an encoder's states, with K-FAC on its four projections.

    y = x + dropout(o(attention(rope(q(x)), rope(k(e)), v(e))))

x: decoder states [batch, len_q, width], e: padded encoder states [batch, len_kv, width] of
kv_len[b] valid rows each.  The projections are torch products; everything between them -
rotary positions, cross attention and dropout with the residual, forward and backward - are the
package's block operators, and their inputs and output gradients are what Kfac's factor updates
take.  k and v read the same input, so their A factor is shared (tie_a_factor).

    python examples/cross_attention_block.py [--steps N]
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

Q, KEY, V, O = range(4)


class Block:
    """fp32 weights [out, in] of the four projections; bf16 activations."""

    def __init__(self, width, heads, kv_heads, batch, len_q, len_kv, seed=0, p=0.1, lr=2e-2,
                 damping=1e-2):
        assert width % heads == 0 and heads % kv_heads == 0
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.dim, self.heads, self.kv_heads, self.p, self.seed = width // heads, heads, kv_heads, p, seed
        kv_width = kv_heads * self.dim
        self.out = [width, kv_width, kv_width, width]
        self.w = [torch.randn(o, width, generator=gen, device="cuda") * width ** -0.5 for o in self.out]
        self.table = K.rope_table(max(len_q, len_kv), self.dim)
        rows = batch * max(len_q, len_kv)
        self.kfac = K.Kfac([(K.KFAC_KRON, o, width, 0, K.KFAC_BF16) for o in self.out],
                           max_rows=rows, lr=lr, damping=damping, momentum=0.9, weight_decay=0.0)
        self.kfac.tie_a_factor(V, KEY)
        self.step_count = 0

    def forward(self, x, e, kv_len):
        b, n, width = x.shape
        w = [t.bfloat16() for t in self.w]
        q = (x @ w[Q].t()).view(b, n, self.heads, self.dim)
        k = (e @ w[KEY].t()).view(b, e.shape[1], self.kv_heads, self.dim)
        v = (e @ w[V].t()).view(b, e.shape[1], self.kv_heads, self.dim)
        K.rope(q, None, self.table, out_q=q)   # in place; queries and keys have lengths of
        K.rope(None, k, self.table, out_k=k)   # their own
        a, lse = K.cross_attention(q, k, v, kv_len=kv_len)
        h = a.view(b, n, width) @ w[O].t()
        y = K.dropout(h, self.p, self.seed, offset=self.step_count, residual=x)
        self.saved = (x, e, kv_len, q, k, v, a, lse, w)
        return y

    def backward(self, dy):
        """Output gradients of the four projections (and the inputs they belong to)."""
        x, e, kv_len, q, k, v, a, lse, w = self.saved
        dh = K.dropout_backward(dy, self.p, self.seed, offset=self.step_count)
        da = (dh @ w[O]).view_as(a)
        dq, dk, dv = K.cross_attention_backward(da, q, k, v, a, lse, kv_len=kv_len)
        K.rope(dq, None, self.table, inverse=True, out_q=dq)
        K.rope(None, dk, self.table, inverse=True, out_k=dk)
        flat = lambda t: t.reshape(-1, t.shape[2] * t.shape[3] if t.dim() == 4 else t.shape[2])
        return [flat(t) for t in (x, e, e, a)], [flat(t) for t in (dq, dk, dv, dh)]

    def step(self, x, e, kv_len, target, refresh_every=5):
        """One K-FAC step on mean((y - target)^2); returns the loss (a device scalar)."""
        y = self.forward(x, e, kv_len)
        d = y.float() - target.float()
        rows = d.shape[0] * d.shape[1]
        dy = (d * (2.0 / d.shape[2])).to(y.dtype)   # per row; the mean over rows is below
        inputs, grads = self.backward(dy)
        for i in range(4):
            tied = i == V
            self.kfac.update_factors(i, None if tied else inputs[i], grads[i])
        if self.step_count % refresh_every == 0:
            self.kfac.invert()
        for i in range(4):
            g = (grads[i].t().float() @ inputs[i].float()) / rows
            self.kfac.precondition(i, g, None, None, None, self.w[i], None)
        self.step_count += 1
        return (d * d).mean()


def train(steps=30, batch=4, len_q=96, len_kv=160, width=256, heads=4, kv_heads=2, seed=0):
    """Fit the block to the output of another of the same shape; returns the losses."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed + 1)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()
    x, e = draw(batch, len_q, width), draw(batch, len_kv, width)
    kv_len = torch.tensor([len_kv * (i + 1) // batch for i in range(batch)], device="cuda",
                          dtype=torch.int32)
    teacher = Block(width, heads, kv_heads, batch, len_q, len_kv, seed=seed + 2, p=0.0)
    target = teacher.forward(x, e, kv_len)
    student = Block(width, heads, kv_heads, batch, len_q, len_kv, seed=seed, p=0.1)
    losses = [student.step(x, e, kv_len, target) for _ in range(steps)]
    code, layer, info = student.kfac.get_status()
    assert code == 0, (code, layer, info)
    assert K.operator_status()[0] == 0
    return [float(l) for l in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    ls = train(a.steps)
    for i, l in enumerate(ls):
        if i % max(1, len(ls) // 10) == 0 or i == len(ls) - 1:
            print(f"step {i:4d}  loss {l:.5f}")
