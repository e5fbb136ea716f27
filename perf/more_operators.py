"""Cases of the operators for the parts of a transformer that have no Kronecker factors: the
orthogonalised update of a weight matrix (Newton-Schulz products), the root-mean-square norm with
the residual's addition and its gradients, the token embedding and its gradient.

A case is a dict of plain values.  prepare() makes its inputs from the seed, run() makes one pass
(own: the library's calls; otherwise elementary torch operations in 32 bits), work() counts the
bytes and operations the pass cannot do without, exact() gives the outputs in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}
_SIZE = {BF16: 2, F32: 4}

# the quintic x -> a x + b x^3 + c x^5 that moves every singular value to about one, five times
A, B, C = 3.4445, -4.7750, 2.0315
STEPS, EPS = 5, 1e-7

# weight matrices [out, in] of the layer sets: one transformer block (width 2048, inner 8192) and
# the MLP
BLOCK = "2048x2048,2048x2048,2048x2048,2048x2048,8192x2048,2048x8192"
MLP = "1024x1024,1024x1024,1024x1024,10x1024"


# ----------------------------------------------------------------------------------- cases

def listed():
    return [
        # the updates of all four blocks of the transformer set, bf16
        _ortho("ortho_transformer_bf16", "direction", BF16, ",".join([BLOCK] * 4)),
        # one odd-sized projection by itself: few tiles, latency
        _ortho("ortho_single_bf16", "direction", BF16, "1000x513"),
        # the MLP set's whole step in fp32: momentum, direction, weights in place
        _ortho("ortho_step_mlp_f32", "step", F32, MLP),
        # the norm before a projection of that block, in training: residual added, forward and
        # backward, the residual stream's gradient joined
        _norm("norm_train_bf16", "train", BF16, 16384, 2048, True, 0),
        # the same in fp32 at a ragged size, no residual
        _norm("norm_train_f32", "train", F32, 4099, 1025, False, 0),
        # a prompt's norm handed to 8-bit products: one scale per 128 channels
        _norm("norm_8bit_bf16", "8bit", BF16, 1920, 2048, True, 128),
        # one new token of each of 16 sequences: latency
        _norm("norm_token_bf16", "forward", BF16, 16, 2048, True, 0),
        # the transformer set's tokens looked up, and the gradient of the whole table
        _embed("embed_train_bf16", "train", BF16, 16384, 2048, 50021, 32),
        # fp32 with a small vocabulary, odd width, padded batch
        _embed("embed_train_f32", "train", F32, 4099, 260, 997, 64),
        # one new token of each of 16 sequences: latency
        _embed("embed_token_bf16", "forward", BF16, 16, 2048, 50021, 32),
    ]


def _ortho(name, kind, dtype, shapes):
    return {"name": name, "op": "ortho", "kind": kind, "dtype": dtype, "shapes": shapes}


def _norm(name, kind, dtype, rows, cols, residual, group):
    return {"name": name, "op": "norm", "kind": kind, "dtype": dtype, "rows": rows, "cols": cols,
            "residual": residual, "group": group}


def _embed(name, kind, dtype, tokens, width, vocabulary, id_bits):
    return {"name": name, "op": "embed", "kind": kind, "dtype": dtype, "tokens": tokens,
            "width": width, "vocabulary": vocabulary, "id_bits": id_bits}


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ortho", "norm", "embed"])
    if op == "ortho":
        kind = rng.choice(["direction", "direction", "step"])
        shapes = ["%dx%d" % (_log_int(rng, 16, 4096), _log_int(rng, 16, 4096))
                  for _ in range(rng.choice([1, 1, 2, 5]))]
        c = _ortho("", kind, F32 if kind == "step" else rng.choice([BF16, BF16, F32]),
                   ",".join(shapes))
    elif op == "norm":
        kind = rng.choice(["train", "train", "8bit", "forward"])
        cols = _log_int(rng, 16, 8192)
        if rng.random() < 0.6:
            cols = max(16, cols // 16 * 16)
        rows = max(1, min(_log_int(rng, 1, 16384), (16384 * 2048) // cols))
        if kind == "8bit":
            rows = max(1, min(rows, 3900000 // cols))
        c = _norm("", kind, rng.choice([BF16, BF16, F32]), rows, cols, rng.random() < 0.6,
                  rng.choice([0, 64, 128]) if kind == "8bit" else 0)
    else:
        width = _log_int(rng, 16, 4096)
        if rng.random() < 0.6:
            width = max(16, width // 16 * 16)
        most = (50021 * 2048) // width
        c = _embed("", rng.choice(["train", "train", "forward"]), rng.choice([BF16, BF16, F32]),
                   min(_log_int(rng, 1, 16384), most), width, min(_log_int(rng, 64, 131072), most),
                   rng.choice([32, 64]))
    del c["name"]
    return c


def _shapes(c):
    return [tuple(int(n) for n in s.split("x")) for s in c["shapes"].split(",")]


# ---------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": c}
    if c["op"] == "ortho":
        def gradient(o, i):
            """A few strong directions and noise, of a gradient's size."""
            r = max(1, min(o, i, 512) // 8)
            strong = torch.logspace(0, -1, r, device="cuda")
            return 1e-4 * ((randn(o, r) * strong) @ randn(r, i) / math.sqrt(r) + 0.2 * randn(o, i))

        s["x"] = [gradient(o, i).to(dt) for o, i in _shapes(c)]
        s["workspace"] = None
        if c["kind"] == "step":
            s["momentum"] = [gradient(o, i) * 4 for o, i in _shapes(c)]
            s["weight"] = [randn(o, i) * i ** -0.5 for o, i in _shapes(c)]
        else:
            s["out"] = [torch.empty_like(x) for x in s["x"]]
        return s
    if c["op"] == "norm":
        m, n = c["rows"], c["cols"]
        # a residual stream: channels of different sizes
        size = torch.exp(0.5 * randn(n))
        s["x"] = (randn(m, n) * size).to(dt)
        s["residual"] = (2 * randn(m, n) * size).to(dt) if c["residual"] else None
        s["gain"] = 1 + 0.2 * randn(n)
        s["workspace"] = None
        if c["kind"] == "train":
            s["dout"] = (1e-2 * randn(m, n)).to(dt)
            s["dresidual"] = (1e-2 * randn(m, n)).to(dt) if c["residual"] else None
        return s
    t, v = c["tokens"], c["vocabulary"]
    # frequencies fall with the rank as in text; one token in 32 is padding (id 0)
    weight = 1.0 / (torch.arange(v, device="cuda", dtype=torch.float64) + 2.7)
    upto = torch.cumsum(weight, 0) / weight.sum()
    draws = torch.rand(t, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.searchsorted(upto, draws).clamp_(max=v - 1)
    ids[torch.rand(t, generator=gen, device="cuda") < 1 / 32] = 0
    s["ids"] = ids.to(torch.int64 if c["id_bits"] == 64 else torch.int32)
    s["table"] = (0.02 * randn(v, c["width"])).to(dt)
    s["scale"] = math.sqrt(c["width"])
    s["workspace"] = None
    if c["kind"] == "train":
        s["dout"] = (1e-3 * randn(t, c["width"])).to(dt)
        s["dtable"] = torch.empty(v, c["width"], device="cuda")
        s["frequency"] = torch.empty(v, device="cuda")
    return s


# ------------------------------------------------------------------------------------- run

LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


def run(state):
    if own:
        return {"ortho": _own_ortho, "norm": _own_norm, "embed": _own_embed}[state["case"]["op"]](state)
    return {"ortho": _plain_ortho, "norm": _plain_norm, "embed": _plain_embed}[state["case"]["op"]](state)


def _own_ortho(s):
    import second_order_optimizer_gb300 as K
    if s["workspace"] is None:   # once, as a program would
        s["workspace"] = K.orthogonalize_workspace(s["x"])
    if s["case"]["kind"] == "step":
        K.orthogonal_step(s["x"], s["momentum"], s["weight"], lr=LR, momentum=MOMENTUM,
                          weight_decay=DECAY, workspace=s["workspace"])
        return {"weight": s["weight"], "momentum": s["momentum"]}
    return K.orthogonalize(s["x"], out=s["out"], workspace=s["workspace"])


def _own_norm(s):
    import second_order_optimizer_gb300 as K
    c = s["case"]
    if c["kind"] == "8bit":
        q, scales, h = K.rms_norm_e4m3(s["x"], s["gain"], residual=s["residual"], group=c["group"])
        return {"q": q, "scales": scales} if h is None else {"q": q, "scales": scales, "h": h}
    y, h, rstd = K.rms_norm(s["x"], s["gain"], residual=s["residual"])
    got = {"y": y} if h is None else {"y": y, "h": h}
    if c["kind"] == "train":
        if s["workspace"] is None:
            s["workspace"] = K.rms_norm_workspace(s["x"])
        got["dx"], got["dgain"], got["dgain_square"] = K.rms_norm_backward(
            s["dout"], s["x"] if h is None else h, s["gain"], rstd, dresidual=s["dresidual"],
            square=True, workspace=s["workspace"])
    return got


def _own_embed(s):
    import second_order_optimizer_gb300 as K
    c = s["case"]
    got = {"out": K.embedding(s["ids"], s["table"], scale=s["scale"])}
    if c["kind"] == "train":
        if s["workspace"] is None:
            s["workspace"] = K.embedding_workspace(s["ids"], c["vocabulary"], c["width"])
        K.embedding_backward(s["ids"], s["dout"], c["vocabulary"], scale=s["scale"], padding_id=0,
                             out=s["dtable"], frequency=s["frequency"], workspace=s["workspace"])
        got["dtable"], got["frequency"] = s["dtable"], s["frequency"]
    return got


def _plain_direction(u):
    """Newton-Schulz products of an fp32 matrix over its Frobenius norm."""
    x = u if u.shape[0] <= u.shape[1] else u.t()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    for _ in range(STEPS):
        g = x @ x.t()
        x = A * x + (B * g + C * (g @ g)) @ x
    return x if u.shape[0] <= u.shape[1] else x.t()


def _plain_ortho(s):
    c = s["case"]
    if c["kind"] == "direction":
        return [_plain_direction(x.float()).to(x.dtype) for x in s["x"]]
    for g, m, w in zip(s["x"], s["momentum"], s["weight"]):
        m.mul_(MOMENTUM).add_(g)
        o = _plain_direction(g + MOMENTUM * m)
        w.sub_(LR * (math.sqrt(max(1.0, w.shape[0] / w.shape[1])) * o + DECAY * w))
    return {"weight": s["weight"], "momentum": s["momentum"]}


NORM_EPS, E4M3_MAX = 1e-6, 448.0


def _plain_norm(s):
    c = s["case"]
    dt, m, n = _DT[c["dtype"]], c["rows"], c["cols"]
    h = s["x"].float()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        got["h"] = h.to(dt)
    rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + NORM_EPS)
    y = h * rstd * s["gain"]
    if c["kind"] == "8bit":
        group = c["group"] or n
        pad = -n % group
        v = torch.nn.functional.pad(y, (0, pad)).view(m, -1, group)
        scales = v.abs().amax(dim=2) / E4M3_MAX
        q = v / torch.where(scales > 0, scales, 1.0)[:, :, None]
        got["q"] = q.view(m, n + pad)[:, :n].to(torch.float8_e4m3fn)
        got["scales"] = scales
        return got
    got["y"] = y.to(dt)
    if c["kind"] == "train":
        xhat = (s["x"] if s["residual"] is None else got["h"]).float() * rstd
        dy = s["dout"].float()
        dx = dy * s["gain"]
        dx = rstd * (dx - xhat * (dx * xhat).mean(dim=1, keepdim=True))
        if s["dresidual"] is not None:
            dx = dx + s["dresidual"].float()
        got["dx"] = dx.to(dt)
        each = dy * xhat
        got["dgain"] = each.sum(dim=0)
        got["dgain_square"] = (each * each).mean(dim=0)
    return got


def _plain_embed(s):
    c = s["case"]
    ids = s["ids"].long()
    got = {"out": (s["table"][ids].float() * s["scale"]).to(s["table"].dtype)}
    if c["kind"] == "train":
        kept = ids != 0
        # per row in 32 bits, tokens of a row in their order of addition
        rows = torch.where(kept[:, None], s["dout"].float() * s["scale"], 0.0)
        got["dtable"] = s["dtable"].zero_().index_add_(0, ids, rows)
        got["frequency"] = s["frequency"].zero_().index_add_(0, ids, kept.float() / c["tokens"])
    return got


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    size = _SIZE[c["dtype"]]
    if c["op"] == "ortho":
        bytes_ = flops = 0
        for o, i in _shapes(c):
            s, l = min(o, i), max(o, i)
            # gradient in; direction out, or momentum and weights read and written
            bytes_ += o * i * (size + (16 if c["kind"] == "step" else size))
            # per step: the two symmetric products by their distinct halves, and one whole one
            flops += STEPS * (s * s * l + s * s * s + 2 * s * s * l)
        return {"bytes": bytes_, "flops": flops}
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        bytes_ = n * size * (3 if c["residual"] else 1) + 4 * c["cols"]   # x, residual in, h out
        flops = 4 * n
        if c["kind"] == "8bit":
            groups = -(-c["cols"] // c["group"]) if c["group"] else 1
            bytes_ += n + 4 * c["rows"] * groups
        else:
            bytes_ += n * size
        if c["kind"] == "train":   # read the gradients, the saved rows; write dx and the sums
            bytes_ += n * size * (4 if c["residual"] else 3) + 8 * c["cols"] + 4 * c["rows"]
            flops += 12 * n
        return {"bytes": bytes_, "flops": flops}
    t, w, v = c["tokens"], c["width"], c["vocabulary"]
    bytes_ = t * (c["id_bits"] // 8 + 2 * w * size)
    flops = t * w
    if c["kind"] == "train":
        bytes_ += t * (c["id_bits"] // 8 + w * size) + v * (4 * w + 4)
        flops += 2 * t * w
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"ortho": _exact_ortho, "norm": _exact_norm, "embed": _exact_embed}[case["op"]](case, s)


def _exact_direction(u):
    """The polynomial of each step as a matrix of the small side's size: X_k = P_k X_0 with
    P_(k+1) = (a + b L + c L^2) P_k and L = X_k X_k^T, which commutes with it."""
    x = u.double()
    x = x.t() if x.shape[0] > x.shape[1] else x
    x = x / (torch.sqrt(torch.sum(x * x)) + EPS)
    gram = x @ x.t()
    eye = torch.eye(gram.shape[0], dtype=torch.float64, device="cuda")
    p, l = eye, gram
    for k in range(STEPS):
        f = A * eye + B * l + C * (l @ l)
        p = f if k == 0 else f @ p
        if k + 1 < STEPS:
            l = f @ l @ f
    x = p @ x
    return x.t() if u.shape[0] > u.shape[1] else x


def _exact_ortho(c, s):
    if c["kind"] == "direction":
        return [_exact_direction(x) for x in s["x"]]
    got = {"weight": [], "momentum": []}
    for g, m, w in zip(s["x"], s["momentum"], s["weight"]):
        g, m, w = g.double(), m.double(), w.double()
        m = MOMENTUM * m + g
        o = _exact_direction(g + MOMENTUM * m)
        got["momentum"].append(m)
        got["weight"].append((1 - LR * DECAY) * w - LR * max(1.0, w.shape[0] / w.shape[1]) ** 0.5 * o)
    return got


def _to_e4m3(v):
    """Nearest value with three mantissa bits (ties to even), exponents from -6, at most 448."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6.0)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(c, s):
    f64, m, n = torch.float64, c["rows"], c["cols"]
    h = s["x"].to(f64)
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].to(f64)
        got["h"] = h
    root = torch.sqrt(h.square().sum(dim=1) / n + NORM_EPS)[:, None]
    y = h / root * s["gain"].to(f64)
    if c["kind"] == "8bit":
        group = c["group"] or n
        q, scales = [], []
        for at in range(0, n, group):
            v = y[:, at:at + group]
            top = v.abs().max(dim=1).values
            scales.append(top / E4M3_MAX)
            q.append(_to_e4m3(v * (E4M3_MAX / torch.where(top > 0, top, 1.0))[:, None]))
        got["q"], got["scales"] = torch.cat(q, dim=1), torch.stack(scales, dim=1)
        return got
    got["y"] = y
    if c["kind"] == "train":
        # the backward pass reads the rows as they were stored, and the forward pass's statistic
        saved = (s["x"] if s["residual"] is None else h.to(_DT[c["dtype"]])).to(f64)
        g = s["dout"].to(f64)
        w = g * s["gain"].to(f64)
        dx = w / root - saved * ((w * saved).sum(dim=1, keepdim=True) / (n * root ** 3))
        got["dx"] = dx if s["dresidual"] is None else dx + s["dresidual"].to(f64)
        got["dgain"] = torch.einsum("ij,ij->j", g, saved / root)
        got["dgain_square"] = torch.einsum("ij,ij->j", g * g, (saved / root) ** 2) / m
    return got


def _exact_embed(c, s):
    f64, ids = torch.float64, s["ids"].long()
    got = {"out": torch.nn.functional.embedding(ids, s["table"].to(f64)) * s["scale"]}
    if c["kind"] == "train":
        order = torch.argsort(ids, stable=True)
        found, count = torch.unique_consecutive(ids[order], return_counts=True)
        dt = torch.zeros(c["vocabulary"], c["width"], dtype=f64, device="cuda")
        rows = s["dout"].to(f64)[order]
        dt[found] = torch.segment_reduce(rows, "sum", lengths=count, axis=0) * s["scale"]
        freq = torch.zeros(c["vocabulary"], dtype=f64, device="cuda")
        freq[found] = count.to(f64) / c["tokens"]
        dt[0] = 0
        freq[0] = 0
        got["dtable"], got["frequency"] = dt, freq
    return got
