"""CPU checks of the block operators: the float64 reference against what its definitions fix
(known generator outputs, rotations, differences of the loss), and every refusal of the entry
points that needs no GPU."""
import ctypes

import numpy as np
import pytest

from oracle import block_oracle as B


# ------------------------------------------------------------------------------- the oracle

def test_philox_known_answers():
    """The published test vectors of Philox4x32-10 (zeros, ones, digits of pi)."""
    f = 0xFFFFFFFF
    cases = [((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
             ((f, f, f, f), (f, f), (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
             ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
              (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1))]
    for ctr, key, want in cases:
        assert tuple(B.philox4x32(ctr, key)) == want


@pytest.mark.parametrize("p", [0.0, 0.25, 1.0])
def test_dropout_keeps_its_share_and_its_mean(p):
    x = np.ones(20000)
    y = B.dropout(x, p, 7, 3)
    kept = (y != 0).mean()
    assert abs(kept - (1 - p)) <= 4 * np.sqrt(0.25 / x.size)
    if p < 1:
        assert np.allclose(y[y != 0], 1 / (1 - p))
    assert np.array_equal(B.dropout(x, p, 7, 3), y)
    if 0 < p < 1:
        assert not np.array_equal(B.dropout(x, p, 7, 4), y)
        assert not np.array_equal(B.dropout(x, p, 8, 3), y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_turns_pairs_and_its_inverse_turns_them_back(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 5, 3, 12))
    table = B.rope_table(40, 8)
    pos = rng.integers(0, 40, (2, 5))
    y = B.rope(x, table, pos, interleaved)
    assert np.allclose(B.rope(y, table, pos, interleaved, inverse=True), x)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # scores depend on the distance of two positions alone
    q, k = x[:1, :1, :1], x[:1, 1:2, :1]
    at = lambda t: np.array([[t]])
    dots = [(B.rope(q, table, at(a), interleaved) * B.rope(k, table, at(c), interleaved)).sum()
            for a, c in ((3, 7), (30, 34))]
    assert abs(dots[0] - dots[1]) <= 1e-12 * max(1, abs(dots[0]))


def test_rope_scalings_at_their_limits():
    plain, _ = B.rope_frequencies(64)
    for scaling in ("linear", "ntk", "yarn"):
        f, mag = B.rope_frequencies(64, scaling=scaling, factor=1.0, original_length=4096)
        assert np.allclose(f, plain) and mag == 1.0
    f, mag = B.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert np.isclose(f[0], plain[0]) and np.isclose(f[-1], plain[-1] / 8)
    f, mag = B.rope_frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    assert np.isclose(f[0], plain[0]) and np.isclose(f[-1], plain[-1] / 8) and mag > 1
    assert np.all(np.diff(f) < 0)


def test_attention_gradients_are_differences_of_the_loss():
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal(s) for s in ((2, 3, 4, 5), (2, 6, 2, 5), (2, 6, 2, 5)))
    g = rng.standard_normal(q.shape)
    ok = B.permitted(2, 6, kv_len=[4, 6], key_mask=rng.random((2, 6)) < 0.7)
    ok[1, 0] = True
    dq, dk, dv = B.cross_attention_backward(g, q, k, v, ok)
    loss = lambda: (B.cross_attention(q, k, v, ok)[0] * g).sum()
    for x, dx in ((q, dq), (k, dk), (v, dv)):
        for _ in range(12):
            i = tuple(rng.integers(0, n) for n in x.shape)
            keep, h = x[i], 1e-5
            x[i] = keep + h
            up = loss()
            x[i] = keep - h
            down = loss()
            x[i] = keep
            # central difference: h^2 truncation and 1e-16 / h rounding, both about 1e-10
            assert abs((up - down) / (2 * h) - dx[i]) <= 1e-8


def test_attention_without_permitted_keys_is_zero():
    q, k, v = np.ones((1, 2, 2, 4)), np.full((1, 3, 1, 4), np.nan), np.full((1, 3, 1, 4), np.inf)
    ok = B.permitted(1, 3, kv_len=[0])
    out, lse = B.cross_attention(q, k, v, ok)
    assert (out == 0).all() and np.isneginf(lse).all()
    assert all((t == 0).all() for t in B.cross_attention_backward(q, q, k, v, ok))


def _bf16(x):
    """Rounded to bf16, to nearest even."""
    i = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    i = (i + 0x7FFF + ((i >> 16) & 1)) & 0xFFFF0000
    return i.astype(np.uint32).view(np.float32).astype(np.float64)


@pytest.mark.parametrize("nq,nk,d", [(20, 3100, 64), (700, 1100, 72), (2500, 40, 128), (300, 129, 80)])
def test_gradient_norm_bounds_tell_roundings_from_mistakes(nq, nk, d):
    """Products with P, dS, out and the results rounded to bf16 stay within the bounds; without delta,
    or without the last tile of keys (dq) or of queries (dk, dv), they do not."""
    rng = np.random.default_rng(nq)
    q, g = (_bf16(rng.standard_normal((1, nq, 1, d))) for _ in range(2))
    k, v = (_bf16(rng.standard_normal((1, nk, 1, d))) for _ in range(2))
    ref, bound = B.gradient_norm_bounds(g, q, k, v, np.ones((1, nk), bool))
    out, lse = B.cross_attention(q, k, v, np.ones((1, nk), bool))
    Q, Kk, V, G, scale = q[0, :, 0], k[0, :, 0], v[0, :, 0], g[0, :, 0], d ** -0.5

    def grads(delta=True, keys=nk, queries=nq):
        p = np.exp(scale * Q @ Kk.T - lse[0, 0][:, None])
        dp = G @ V.T
        o = _bf16(out[0, :, 0])
        t = (p * dp).sum(axis=1) if nk <= 128 else (G * o).sum(axis=1)
        ds = _bf16(p * (dp - t[:, None] * delta))
        return (_bf16(scale * ds[:, :keys] @ Kk[:keys]), _bf16(scale * ds[:queries].T @ Q[:queries]),
                _bf16(_bf16(p)[:queries].T @ G[:queries]))

    off = lambda got: [np.linalg.norm(x - y.reshape(x.shape)) / b for x, y, b in zip(
        (r[0, :, 0] for r in ref), got, bound)]
    assert max(off(grads())) <= 1
    assert min(off(grads(delta=False))[:2]) > 1
    if nk > 128:
        assert off(grads(keys=(nk - 1) // 128 * 128))[0] > 1
    if nq > 128:
        assert min(off(grads(queries=(nq - 1) // 128 * 128))[1:]) > 1


# ------------------------------------------------------------- refusals (nothing is launched)

@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import second_order_optimizer_gb300._lib as L
    return L


A, W, U = 1, 2, 7   # KFAC_ERR_INVALID_ARG, KFAC_ERR_WORKSPACE, KFAC_ERR_UNSUPPORTED
P = 0x10000         # an aligned address that is never read


def _rope(lib, q=P, k=P, table=P, pos=None, oq=2 * P, ok=2 * P, **kw):
    d = dict(dtype=1, batch=2, length=4, heads=2, kv_heads=1, head_dim=16, rotary_dim=8,
             interleaved=0, inverse=0, table_rows=64, position_offset=0, position_stride=4,
             qs=(128, 32, 16), ks=(64, 16, 16), oqs=(128, 32, 16), oks=(64, 16, 16))
    d.update(kw)
    s = [d.pop(n) for n in ("qs", "ks", "oqs", "oks")]
    desc = lib.ROPE_DESC.pack(*d.values(), *(x for t in s for x in t))
    return lib.LIB.kfac_rope(desc, q, k, table, pos, oq, ok, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(batch=-1), dict(head_dim=0), dict(rotary_dim=7), dict(rotary_dim=0),
    dict(rotary_dim=18), dict(interleaved=2), dict(inverse=-1), dict(table_rows=0),
    dict(position_offset=-1), dict(position_offset=61), dict(q=None), dict(ok=None), dict(k=P + 1),
    dict(table=None), dict(table=P + 2), dict(pos=P + 2), dict(qs=(-1, 32, 16)),
    dict(oqs=(128, 8, 16)),                       # output rows overlap
    dict(oqs=(0, 32, 16)),                        # an output broadcast over the batch
    dict(oq=P, oqs=(256, 32, 16))])               # in place with other strides
def test_rope_refuses(lib, kw):
    assert _rope(lib, **kw) == A


def test_rope_table_refuses(lib):
    f = lambda rows=4, r=8, base=1e4, scaling=0, factor=1.0, n=1.0, t=P: lib.LIB.kfac_rope_table(
        t, rows, r, base, scaling, factor, n, None)
    assert [f(t=None), f(rows=-1), f(r=3), f(r=0), f(base=1.0), f(base=float("nan")),
            f(scaling=4), f(scaling=-1), f(scaling=1, factor=0.5),
            f(scaling=3, factor=2.0, n=0.0), f(scaling=2, factor=2.0, r=2)] == [A] * 11
    assert f(rows=0) == 0


def test_dropout_refuses(lib):
    f = lambda dt=0, x=P, ldx=8, r=None, ldr=8, o=P, ldo=8, rows=3, cols=8, p=0.5: (
        lib.LIB.kfac_dropout(dt, x, ldx, r, ldr, o, ldo, rows, cols, p, 1, 0, None))
    assert [f(dt=2), f(x=None), f(o=None), f(x=P + 2), f(r=P + 1), f(ldx=7), f(ldo=0),
            f(r=P, ldr=4), f(rows=-1), f(cols=-1), f(p=-0.1), f(p=1.5), f(p=float("nan"))] == [A] * 13
    assert f(rows=0) == 0 and f(cols=0, x=None) == 0


def _desc(lib, **kw):
    d = dict(dtype=1, batch=2, len_q=4, len_kv=6, heads=4, kv_heads=2, head_dim=16, scale=0.0,
             qs=(256, 64, 16), ks=(192, 32, 16), vs=(192, 32, 16), os=(256, 64, 16))
    d.update(kw)
    s = [d.pop(n) for n in ("qs", "ks", "vs", "os")]
    return lib.ATTENTION_DESC.pack(*d.values(), *(x for t in s for x in t))


BAD_DESC = [dict(dtype=3), dict(batch=-1), dict(len_q=-1), dict(len_kv=-1), dict(heads=0),
            dict(kv_heads=3), dict(kv_heads=0), dict(head_dim=0), dict(scale=-1.0),
            dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("kw", BAD_DESC)
def test_attention_refuses_bad_descriptors(lib, kw):
    n = ctypes.c_size_t(0)
    d, g = _desc(lib, **kw), lib.ATTENTION_GRAD_DESC.pack(*([1024] * 12))
    assert lib.LIB.kfac_cross_attention_workspace_size(d, 0, ctypes.byref(n)) == A
    assert lib.LIB.kfac_cross_attention(d, P, P, P, None, None, P, P, P, 1 << 30, None) == A
    assert lib.LIB.kfac_cross_attention_backward(d, g, P, P, P, P, P, P, None, None, P, P, P, P,
                                                 1 << 30, None) == A


def test_attention_refuses(lib):
    fwd = lambda d=None, q=P, k=P, v=P, n=None, m=None, o=P, lse=P, ws=P, nb=1 << 30: (
        lib.LIB.kfac_cross_attention(d or _desc(lib), q, k, v, n, m, o, lse, ws, nb, None))
    assert [fwd(q=None), fwd(k=None), fwd(v=P + 1), fwd(o=None), fwd(n=P + 2), fwd(lse=P + 2),
            fwd(_desc(lib, os=(256, 8, 16))), fwd(_desc(lib, os=(0, 64, 16))),
            fwd(_desc(lib, ks=(192, -32, 16)))] == [A] * 9
    assert fwd(_desc(lib, head_dim=129, qs=(4096, 1024, 256), os=(4096, 1024, 256))) == U
    assert fwd(_desc(lib, batch=0)) == 0 and fwd(_desc(lib, len_q=0)) == 0
    grads = lambda **kw: lib.ATTENTION_GRAD_DESC.pack(*(x for n, s in (
        ("dout", (256, 64, 16)), ("dq", (256, 64, 16)), ("dk", (192, 32, 16)),
        ("dv", (192, 32, 16))) for x in kw.get(n, s)))
    bwd = lambda d=None, g=None, do=P, lse=P, dq=P, dk=P, dv=P, ws=P, nb=1 << 30: (
        lib.LIB.kfac_cross_attention_backward(d or _desc(lib), g or grads(), do, P, P, P, P, lse,
                                              None, None, dq, dk, dv, ws, nb, None))
    assert [bwd(do=None), bwd(lse=None), bwd(lse=P + 1), bwd(dq=None), bwd(dk=P + 1),
            bwd(dv=None), bwd(g=grads(dk=(0, 32, 16))), bwd(g=grads(dq=(256, 64, 8)))] == [A] * 8
    assert lib.LIB.kfac_cross_attention_backward(_desc(lib), None, P, P, P, P, P, P, None, None,
                                                 P, P, P, P, 1 << 30, None) == A
    assert [bwd(ws=None), bwd(ws=P + 16), bwd(nb=16)] == [W] * 3


def test_attention_workspace_is_what_the_backward_pass_needs(lib):
    n = ctypes.c_size_t(0)
    d = _desc(lib)
    assert lib.LIB.kfac_cross_attention_workspace_size(d, 1, ctypes.byref(n)) == 0
    assert n.value % 256 == 0 and n.value >= 2 * 4 * 4 * 4   # one fp32 statistic per query row
    assert lib.LIB.kfac_cross_attention_workspace_size(d, 2, ctypes.byref(n)) == A
    assert lib.LIB.kfac_cross_attention_workspace_size(d, 0, None) == A
    assert lib.LIB.kfac_cross_attention_workspace_size(None, 0, ctypes.byref(n)) == A


def test_python_refuses_cpu_tensors_and_wrong_types(lib):
    torch = pytest.importorskip("torch")
    import second_order_optimizer_gb300 as K
    x = torch.zeros(2, 3, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        K.rope(x, None, torch.zeros(3, 8))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        K.dropout(x.double(), 0.5, 1)
    with pytest.raises(ValueError, match="CUDA"):
        K.dropout(x, 0.5, 1)
    with pytest.raises(ValueError, match="64-bit"):
        K.dropout(x, 0.5, -1)
    with pytest.raises(ValueError, match="CUDA"):
        K.cross_attention(x, x, x)


def test_python_refuses_a_scale_that_would_mean_the_default(lib):
    """The library takes a scale of 0 for 1/sqrt(head_dim): a caller's own 0, or what rounds to 0,
    may not become that."""
    torch = pytest.importorskip("torch")
    from second_order_optimizer_gb300 import _block
    x = torch.zeros(2, 3, 4, 16)
    desc = lambda scale: _block._attention("attention", x, x, x, x, scale, -1)
    for scale in (0.0, 0, -0.0, 1e-50, 1e39, -1e300):
        with pytest.raises(ValueError, match="scale"):
            desc(scale)
    at = lib.struct.calcsize("@7i")
    assert [lib.struct.unpack_from("f", desc(x), at)[0] for x in (None, 0.25, 2.0 ** -126)] == [0.0, 0.25, 2.0 ** -126]
    n = ctypes.c_size_t(0)
    for scale in (-1.0, float("nan"), float("inf")):   # refused by the library
        assert lib.LIB.kfac_cross_attention_workspace_size(desc(scale), 0, ctypes.byref(n)) == A


# ------------------------------------------------------------------- state kept per device

def test_shared_memory_limits_are_set_on_every_device(tmp_path):
    """The helper behind the attention launches, compiled for the host with a call that counts:
    once per device, again where it failed, and past the devices it has room for every time.  No
    launch keeps a flag of its own for the whole process."""
    import os
    import re
    import shutil
    import subprocess
    import __graft_entry__
    csrc = os.path.join(__graft_entry__.ROOT, "second_order_optimizer_gb300", "csrc")
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "t.cpp"
    src.write_text("""
#include "per_device.h"
int main() {
  static kfac::OncePerDevice once;
  int calls[3] = {0, 0, 0};
  bool works = true;
  auto set = [&](int d) { return once(d, [&] { ++calls[d % 3]; return works; }); };
  if (!set(0) || !set(0) || calls[0] != 1) return 1;
  if (!set(1) || calls[1] != 1) return 2;          // another device: set there too
  works = false;
  if (set(2) || set(2) || calls[2] != 2) return 3; // a failure is not remembered
  works = true;
  if (!set(2) || !set(2) || calls[2] != 3) return 4;
  if (!set(99) || !set(99) || calls[0] != 3) return 5;
  return 0;
}
""")
    subprocess.run([gxx, "-std=c++17", "-I" + csrc, str(src), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")]).returncode == 0
    for name in sorted(os.listdir(csrc)):
        if name.startswith(("attn", "k_attn")):
            text = open(os.path.join(csrc, name)).read()
            assert not re.search(r"static\s+const\s+bool\s+\w+\s*=", text), name
            assert text.count("cudaFuncSetAttribute(") == (name == "attn.cuh"), name


def test_rings_wait_for_the_last_copy_of_every_slot(tmp_path):
    """A block that gives up may not end while copies into its shared memory are under way.  Every
    count of issued tiles and every landed part of them, against a model of the slots' barriers
    (phase c has begun once c copies have landed; a wait for parity p ends unless phase c with
    c % 2 == p is the present one): the wait ends exactly when the slot's last copy has landed.  The
    parity of the tile at which the producer stopped, for every slot, does not do that."""
    import os
    import shutil
    import subprocess
    import __graft_entry__
    csrc = os.path.join(__graft_entry__.ROOT, "second_order_optimizer_gb300", "csrc")
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "t.cpp"
    src.write_text("""
#include "ring.h"
int main() {
  bool other_fails = false;
  for (int stages = 1; stages <= 4; ++stages)
    for (int issued = 0; issued <= 40; ++issued) {
      int all = 0;
      for (int s = 0; s < stages; ++s) {
        int uses = 0;
        for (int i = 0; i < issued; ++i) uses += i % stages == s;
        if (kfac::ring_uses(issued, s, stages) != uses) return 1;
        all += uses;
        for (int landed = uses > 0 ? uses - 1 : 0; landed <= uses && uses > 0; ++landed) {
          auto ends = [&](unsigned parity) { return (unsigned)(landed & 1) != parity; };
          if (ends(kfac::ring_last_parity(uses)) != (landed == uses)) return 2;
          other_fails |= ends((unsigned)(issued / stages) & 1u) != (landed == uses);
        }
      }
      if (all != issued) return 3;
    }
  return other_fails ? 0 : 4;
}
""")
    subprocess.run([gxx, "-std=c++17", "-I" + csrc, str(src), "-o", str(tmp_path / "t")], check=True)
    assert subprocess.run([str(tmp_path / "t")]).returncode == 0
