"""Cases of the operators between a decoder block's linear layers: rotary positions, cross
attention to an encoder's states (forward, forward and backward, single tokens), and dropout
with the residual added.

A case is a dict of plain values.  prepare() makes its inputs from the seed, run() makes one
pass (own: the library's calls; otherwise elementary torch operations in 32 bits), work() counts
the bytes and operations the pass cannot do without, exact() gives the outputs in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
_DT = {BF16: torch.bfloat16, F32: torch.float32}


# ----------------------------------------------------------------------------------- cases

def listed():
    return [
        # q and k of one block of the transformer layer set (16384 tokens, width 2048), forward
        _rope("rope_block_bf16", BF16, 8, 2048, 16, 16, 128, 128, False, False, "rows", 2048),
        # gradients of packed sequences: fp32, interleaved pairs, a part of an odd-sized head
        # rotated, shared key heads, positions given per token
        _rope("rope_backward_f32_part", F32, 3, 1021, 12, 4, 80, 32, True, True, "given", 4096),
        # one new token of each of 16 sequences far out in a long scaled context
        _rope("rope_token_bf16", BF16, 16, 1, 16, 4, 128, 128, False, False, "given", 131072),
        # the output projection of that block, dropped and added to the residual stream
        _drop("dropout_block_bf16", BF16, 16384, 2048, 0.1, True, False),
        # its backward form in fp32 at a ragged size
        _drop("dropout_backward_f32", F32, 4099, 1025, 0.25, False, True),
        # a micro-batch of a few rows: latency
        _drop("dropout_small_bf16", BF16, 16, 2048, 0.1, True, False),
        # a training step of that block reading encoder states twice its length, padded
        _attn("attention_train_bf16", BF16, "train", 8, 2048, 4096, 16, 16, 128, "ragged"),
        # training with shared key heads, odd lengths, padding scattered among the keys and one
        # sequence without any encoder state
        _attn("attention_train_gqa_d64", BF16, "train", 5, 577, 1531, 16, 4, 64, "holes"),
        # training in fp32 at odd lengths
        _attn("attention_train_f32", F32, "train", 2, 257, 515, 8, 8, 64, "ragged"),
        # a prompt read against long encoder states, no gradient
        _attn("attention_prompt_bf16", BF16, "forward", 4, 1000, 8192, 16, 4, 128, "ragged"),
        # one new token of each of 32 sequences against long encoder states
        _attn("attention_token_bf16", BF16, "token", 32, 1, 8192, 16, 4, 128, "ragged"),
        # one new token of one short sequence: latency
        _attn("attention_token_small", BF16, "token", 1, 1, 333, 16, 16, 64, "full"),
    ]


def _rope(name, dtype, batch, length, heads, kv_heads, dim, rotary, interleaved, inverse,
          positions, table):
    return {"name": name, "op": "rope", "dtype": dtype, "batch": batch, "length": length,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "inverse": inverse, "positions": positions,
            "table": table}


def _drop(name, dtype, rows, cols, p, residual, backward):
    return {"name": name, "op": "dropout", "dtype": dtype, "rows": rows, "cols": cols, "p": p,
            "residual": residual, "backward": backward}


def _attn(name, dtype, kind, batch, len_q, len_kv, heads, kv_heads, dim, keys):
    return {"name": name, "op": "attention", "dtype": dtype, "kind": kind, "batch": batch,
            "len_q": len_q, "len_kv": len_kv, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "keys": keys}


def _log_int(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "dropout", "attention", "attention"])
    dtype = rng.choice([BF16, BF16, F32])
    if op == "dropout":
        rows, cols = _log_int(rng, 1, 16384), _log_int(rng, 33, 4097)
        c = _drop("", dtype, rows, cols, rng.choice([0.05, 0.1, 0.25, 0.5]),
                  rng.random() < 0.6, rng.random() < 0.4)
        c["residual"] = c["residual"] and not c["backward"]
    elif op == "rope":
        dim = rng.choice([32, 64, 80, 96, 128])
        tokens, length = _log_int(rng, 1, 16384), _log_int(rng, 1, 2048)
        kv = rng.choice([1, 2, 4, 8])
        c = _rope("", dtype, max(1, tokens // length), length, kv * rng.choice([1, 2, 4]), kv, dim,
                  rng.choice([dim, dim // 2, dim // 4]), rng.random() < 0.5, rng.random() < 0.5,
                  rng.choice(["rows", "given"]), _log_int(rng, max(length, 64), 131072))
    else:
        kind = rng.choice(["train", "forward", "token"])
        dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 36])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4])
        batch = _log_int(rng, 1, 32)
        len_q = rng.choice([1, 1, 2, 5, 8]) if kind == "token" else _log_int(rng, 9, 2049)
        len_kv = _log_int(rng, 1, 8193)
        # at most a tenth of the largest listed case in operations (a hundredth in fp32, and where
        # the head's rows are not whole 16 bytes: these run on the CUDA cores)
        most = 2.0e11 if dtype == BF16 and dim % 8 == 0 else 2.0e10
        each = (14 if kind == "train" else 4) * kv * group * dim * len_q * len_kv
        batch = max(1, min(batch, int(most / each)))
        if each > most:
            len_kv = max(1, int(len_kv * most / each))
        c = _attn("", dtype, kind, batch, len_q, len_kv, kv * group, kv, dim,
                  rng.choice(["full", "ragged", "holes"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------- inputs

def _lengths(c):
    """Permitted keys of each sequence, before prepare() permutes them."""
    b, n = c["batch"], c["len_kv"]
    return [max(1, (n * (i + 1)) // b) for i in range(b)]


def _holes(c):
    """Of each sequence's keys, the number that is permitted: four fifths, and none of the
    first sequence's where there are several."""
    b, n = c["batch"], c["len_kv"]
    return [0 if b > 1 and i == 0 else max(1, (4 * n) // 5) for i in range(b)]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DT[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dt)

    s = {"case": c}
    if c["op"] == "dropout":
        s["x"] = randn(c["rows"], c["cols"])
        s["residual"] = randn(c["rows"], c["cols"]) if c["residual"] else None
        s["out"] = torch.empty_like(s["x"])
        s["seed"], s["offset"] = 1_000_003 * int(seed) + 17, int(seed) % 1000
        return s
    if c["op"] == "rope":
        b, n, d, r = c["batch"], c["length"], c["dim"], c["rotary"]
        s["q"], s["k"] = randn(b, n, c["heads"], d), randn(b, n, c["kv_heads"], d)
        s["out_q"], s["out_k"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        # cosines and sines of every position, angles in 64 bits; contexts over 4096 by linear
        # interpolation to that length
        f = 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        f = f / max(1.0, c["table"] / 4096)
        angle = torch.arange(c["table"], device="cuda", dtype=torch.float64)[:, None] * f[None, :]
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["positions"] = None
        if c["positions"] == "given":
            s["positions"] = torch.randint(0, c["table"], (b, n), generator=gen, device="cuda",
                                           dtype=torch.int32)
        return s
    b, nq, nk, h, kv, d = (c[x] for x in ("batch", "len_q", "len_kv", "heads", "kv_heads", "dim"))
    s["q"], s["k"], s["v"] = randn(b, nq, h, d), randn(b, nk, kv, d), randn(b, nk, kv, d)
    s["kv_len"] = s["key_mask"] = None
    if c["keys"] == "ragged":
        order = torch.randperm(b, generator=gen, device="cuda")
        s["kv_len"] = torch.tensor(_lengths(c), device="cuda", dtype=torch.int32)[order]
    elif c["keys"] == "holes":
        most = torch.tensor(_holes(c), device="cuda")
        rank = torch.rand(b, nk, generator=gen, device="cuda").argsort(dim=1).argsort(dim=1)
        s["key_mask"] = (rank < most[:, None]).to(torch.uint8)
        # what stands in padded places is whatever was there
        bad = s["key_mask"] == 0
        s["k"][bad], s["v"][bad] = float("nan"), float("inf")
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(b, h, nq, device="cuda")
    s["workspace"] = None
    if c["kind"] == "train":
        s["dout"] = randn(b, nq, h, d)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
    return s


# ------------------------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "dropout": _own_dropout, "attention": _own_attention}[op](state)
    return {"rope": _plain_rope, "dropout": _plain_dropout,
            "attention": _plain_attention}[op](state)


def _own_rope(s):
    import second_order_optimizer_gb300 as K
    c = s["case"]
    K.rope(s["q"], s["k"], s["table"], positions=s["positions"], interleaved=c["interleaved"],
           inverse=c["inverse"], out_q=s["out_q"], out_k=s["out_k"])
    return {"q": s["out_q"], "k": s["out_k"]}


def _own_dropout(s):
    import second_order_optimizer_gb300 as K
    c = s["case"]
    if c["backward"]:
        return K.dropout_backward(s["x"], c["p"], s["seed"], s["offset"], out=s["out"])
    return K.dropout(s["x"], c["p"], s["seed"], s["offset"], residual=s["residual"], out=s["out"])


def _own_attention(s):
    import second_order_optimizer_gb300 as K
    train = s["case"]["kind"] == "train"
    if s["workspace"] is None:   # once, as a program would
        s["workspace"] = K.cross_attention_workspace(s["q"], s["k"], backward=train)
    K.cross_attention(s["q"], s["k"], s["v"], kv_len=s["kv_len"], key_mask=s["key_mask"],
                      out=s["out"], lse=s["lse"], workspace=s["workspace"])
    got = {"out": s["out"], "lse": s["lse"]}
    if train:
        K.cross_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                   kv_len=s["kv_len"], key_mask=s["key_mask"], dq=s["dq"],
                                   dk=s["dk"], dv=s["dv"], workspace=s["workspace"])
        got.update(dq=s["dq"], dk=s["dk"], dv=s["dv"])
    return got


def _plain_rope(s):
    c = s["case"]
    r, n = c["rotary"], c["length"]
    if s["positions"] is None:
        rows = s["table"][:n].view(1, n, 1, r)
    else:
        rows = s["table"][s["positions"].long()][:, :, None, :]
    cos, sin = rows[..., :r // 2], rows[..., r // 2:]
    if c["inverse"]:
        sin = -sin

    def turn(x):
        x = x.float()
        if c["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            y = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            y = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([y, x[..., r:]], dim=-1).to(_DT[c["dtype"]])

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _plain_dropout(s):
    """Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011) in
    64-bit integers: counter words (i / 4, offset), key = seed, word i mod 4 for element i."""
    c = s["case"]
    x = s["x"]
    low = 0xFFFFFFFF
    count = (x.numel() + 3) // 4
    i = torch.arange(count, device=x.device)
    c0, c1 = i & low, i >> 32
    c2, c3 = torch.full_like(i, s["offset"] & low), torch.full_like(i, s["offset"] >> 32)
    k0, k1 = s["seed"] & low, (s["seed"] >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57   # the low 64 bits, whatever their sign
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    u = torch.stack([c0, c1, c2, c3], dim=1).flatten()[:x.numel()].view(x.shape)
    keep = u >= int(c["p"] * 4294967296.0)
    y = torch.where(keep, x.float() * (1.0 / (1.0 - c["p"])), torch.zeros((), device=x.device))
    if s["residual"] is not None:
        y = s["residual"].float() + y
    return y.to(x.dtype)


def _permitted(s):
    """[batch, len_kv]: whether a key is permitted."""
    c = s["case"]
    if s["key_mask"] is not None:
        return s["key_mask"] != 0
    at = torch.arange(c["len_kv"], device="cuda")[None, :]
    if s["kv_len"] is None:
        return (at >= 0).expand(c["batch"], -1)
    return at < s["kv_len"][:, None]


def _plain_attention(s):
    c = s["case"]
    b, nq, nk, h, kv, d = (c[x] for x in ("batch", "len_q", "len_kv", "heads", "kv_heads", "dim"))
    g, scale, dt = h // kv, 1.0 / math.sqrt(d), _DT[c["dtype"]]
    ok = _permitted(s)
    zero = torch.zeros((), device="cuda")
    # [b, kv, g nq, d] against [b, kv, nk, d]
    heads = lambda x: x.float().view(b, nq, kv, g, d).permute(0, 2, 3, 1, 4).reshape(b, kv, g * nq, d)
    keys = lambda x: torch.where(ok[:, :, None, None], x.float(), zero).transpose(1, 2)
    q, k, v = heads(s["q"]), keys(s["k"]), keys(s["v"])
    back = lambda x: x.view(b, kv, g, nq, d).permute(0, 3, 1, 2, 4).reshape(b, nq, h, d)
    scores = torch.where(ok[:, None, None, :], (q @ k.transpose(2, 3)) * scale, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, zero, top))
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(total)).view(b, h, nq)
    p = p / torch.where(total == 0, 1.0, total)
    out = p @ v
    got = {"out": back(out).to(dt), "lse": lse}
    if c["kind"] == "train":
        do = heads(s["dout"])
        dv = p.transpose(2, 3) @ do
        dp = do @ v.transpose(2, 3)
        ds = p * (dp - (do * out).sum(dim=-1, keepdim=True))
        got["dq"] = back((ds @ k) * scale).to(dt)
        got["dk"] = ((ds.transpose(2, 3) @ q) * scale).transpose(1, 2).to(dt)
        got["dv"] = dv.transpose(1, 2).to(dt)
    return got


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    size = 2 if c["dtype"] == BF16 else 4
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": n * size * (3 if c["residual"] else 2), "flops": 2 * n}
    if c["op"] == "rope":
        tokens = c["batch"] * c["length"]
        rows = c["length"] if c["positions"] == "rows" else min(tokens, c["table"])
        n = tokens * (c["heads"] + c["kv_heads"])
        given = 4 * tokens if c["positions"] == "given" else 0
        return {"bytes": 2 * n * c["dim"] * size + 4 * rows * c["rotary"] + given,
                "flops": 3 * n * c["rotary"]}
    b, nq, nk, h, kv, d = (c[x] for x in ("batch", "len_q", "len_kv", "heads", "kv_heads", "dim"))
    pairs = sum({"full": [nk] * b, "ragged": _lengths(c), "holes": _holes(c)}[c["keys"]])
    q, k = b * nq * h * d * size, pairs * kv * d * size
    extra = {"full": 0, "ragged": 4 * b, "holes": b * nk}[c["keys"]]
    bytes_, flops = 2 * q + 2 * k + 4 * b * h * nq + extra, 4 * h * d * nq * pairs
    if c["kind"] == "train":   # the gradients: read dout, write dq, dk, dv (whole)
        bytes_ += 2 * q + 2 * b * nk * kv * d * size
        flops += 10 * h * d * nq * pairs
    return {"bytes": bytes_, "flops": flops}


# ----------------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "dropout": _exact_dropout, "attention": _exact_attention}[
        case["op"]](case, s)


def _exact_rope(c, s):
    """Each pair as a complex number times exp(+-i angle)."""
    r = c["rotary"]
    t = s["table"].double()
    turn = torch.complex(t[:, :r // 2], t[:, r // 2:])
    turn = turn.conj().resolve_conj() if c["inverse"] else turn
    at = s["positions"].long() if s["positions"] is not None else (
        torch.arange(c["length"], device="cuda").expand(c["batch"], -1))
    turn = turn[at].unsqueeze(2)
    got = {}
    for name in "qk":
        x = s[name].double()
        y = x.clone()
        first = slice(0, r, 2) if c["interleaved"] else slice(0, r // 2)
        second = slice(1, r, 2) if c["interleaved"] else slice(r // 2, r)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        got[name] = y
    return got


def _exact_dropout(c, s):
    n = c["rows"] * c["cols"]
    u32, u64 = np.uint32, np.uint64
    i = np.arange((n + 3) // 4, dtype=u64)
    ctr = [i.astype(u32), (i >> u64(32)).astype(u32),
           np.full(i.shape, s["offset"] & 0xFFFFFFFF, u32), np.full(i.shape, s["offset"] >> 32, u32)]
    key = [s["seed"] & 0xFFFFFFFF, (s["seed"] >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        a = ctr[0].astype(u64) * u64(0xD2511F53)
        b = ctr[2].astype(u64) * u64(0xCD9E8D57)
        ctr = [(b >> u64(32)).astype(u32) ^ ctr[1] ^ u32(key[0]), b.astype(u32),
               (a >> u64(32)).astype(u32) ^ ctr[3] ^ u32(key[1]), a.astype(u32)]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    u = np.stack(ctr, axis=1).reshape(-1)[:n].reshape(c["rows"], c["cols"])
    keep = u.astype(np.float64) >= math.floor(c["p"] * 2.0 ** 32)
    y = np.where(keep, s["x"].double().cpu().numpy() / (1.0 - c["p"]), 0.0)
    return y if s["residual"] is None else y + s["residual"].double().cpu().numpy()


def _exact_attention(c, s):
    """One sequence and key head at a time: softmax over the permitted keys alone, gradients by
    differentiating it."""
    b, nq, nk, h, kv, d = (c[x] for x in ("batch", "len_q", "len_kv", "heads", "kv_heads", "dim"))
    g, f64 = h // kv, torch.float64
    train = c["kind"] == "train"
    zeros = lambda *n: torch.zeros(*n, device="cuda", dtype=f64)
    got = {"out": zeros(b, nq, h, d), "lse": torch.full((b, h, nq), -math.inf, device="cuda", dtype=f64)}
    if train:
        got.update(dq=zeros(b, nq, h, d), dk=zeros(b, nk, kv, d), dv=zeros(b, nk, kv, d))
    for i in range(b):
        at = torch.arange(nk, device="cuda")
        if s["kv_len"] is not None:
            at = at[:int(s["kv_len"][i])]
        if s["key_mask"] is not None:
            at = at[s["key_mask"][i] != 0]
        if at.numel() == 0:
            continue
        for j in range(kv):
            mine = slice(j * g, (j + 1) * g)
            q = s["q"][i, :, mine].to(f64).transpose(0, 1).contiguous().requires_grad_(train)
            k = s["k"][i, at, j].to(f64).requires_grad_(train)
            v = s["v"][i, at, j].to(f64).requires_grad_(train)
            z = torch.matmul(q, k.t()) / d ** 0.5
            o = torch.matmul(torch.softmax(z, dim=-1), v)
            got["out"][i, :, mine] = o.detach().transpose(0, 1)
            got["lse"][i, mine] = torch.logsumexp(z.detach(), dim=-1)
            if train:
                do = s["dout"][i, :, mine].to(f64).transpose(0, 1)
                dq, dk, dv = torch.autograd.grad(o, (q, k, v), do)
                got["dq"][i, :, mine] = dq.transpose(0, 1)
                got["dk"][i, at, j], got["dv"][i, at, j] = dk, dv
    return got
