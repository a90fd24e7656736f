"""Linear attention and rotary positions, what needs no GPU: the reference against closed forms
and differences, argument checks of the C ABI and of the binding, workspace sizes."""
import ctypes
import math

import pytest
import torch

import linattn_ref as ref
from linear_rnn_ckda_b200 import build as lib_build
from linear_rnn_ckda_b200 import ops


@pytest.fixture(scope="module")
def lib():
    lib_build.build_library()
    return ops.load()


def rnd(*shape, seed=0, dtype=torch.float64):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(dtype)


def test_reference_closed_forms():
    """One token: o = (q.k) v + e^g q S0; no decay and one-hot keys: sums of values; g = -inf: a reset."""
    q, k, v = rnd(1, 1, 1, 4, seed=1), rnd(1, 1, 1, 4, seed=2), rnd(1, 1, 1, 3, seed=3)
    S0, g = rnd(1, 1, 4, 3, seed=4), torch.tensor([[[-0.5]]], dtype=torch.float64)
    o, S = ref.fwd(q, k, v, g, S0)
    want = (q[0, 0, 0] @ k[0, 0, 0]) * v[0, 0, 0] + math.exp(-0.5) * (q[0, 0, 0] @ S0[0, 0])
    assert torch.allclose(o[0, 0, 0], want, atol=1e-14)
    T = 5
    one = torch.zeros(1, T, 1, 4, dtype=torch.float64)
    one[..., 2] = 1
    v = rnd(1, T, 1, 3, seed=5)
    o, _ = ref.fwd(one, one, v, torch.zeros(1, dtype=torch.float64))
    assert torch.allclose(o[0, :, 0], v[0, :, 0].cumsum(0), atol=1e-14)
    g = torch.zeros(1, T, 1, dtype=torch.float64)
    g[0, 3] = -math.inf
    o, _ = ref.fwd(one, one, v, g)
    assert torch.allclose(o[0, 3:, 0], v[0, 3:, 0].cumsum(0), atol=1e-14)


@pytest.mark.parametrize("fixed", [False, True])
def test_reference_gradients_by_differences(fixed):
    B, T, H, dk, dv, cu = 1, 7, 4, 3, 2, [0, 3, 3, 7]
    t = dict(q=rnd(B, T, 2, dk, seed=1), k=rnd(B, T, 1, dk, seed=2), v=rnd(B, T, 4, dv, seed=3),
             g=-rnd(H, seed=4).abs() if fixed else -rnd(B, T, H, seed=4).abs(), S0=rnd(3, H, dk, dv, seed=5))
    dO, dS = rnd(B, T, H, dv, seed=6), rnd(3, H, dk, dv, seed=7)

    def loss(**w):
        o, S = ref.fwd(w["q"], w["k"], w["v"], w["g"], w["S0"], cu)
        return float((o * dO).sum() + (S * dS).sum())

    got = dict(zip(("q", "k", "v", "g", "S0"), ref.bwd(**t, cu=cu, dO=dO, dS_T=dS)))
    for name, x in t.items():
        d = rnd(*x.shape, seed=8)
        e = 1e-5
        num = (loss(**{**t, name: x + e * d}) - loss(**{**t, name: x - e * d})) / (2 * e)
        assert abs(num - float((got[name] * d).sum())) < 1e-7 * max(1.0, abs(num)), name


def test_gradient_formulas():
    """The formulas the kernels follow: each of dq, dk, dv is the same recurrence with the roles
    exchanged (dk and dv with time reversed), and dg is a suffix sum of q.dq - k.dk."""
    T, dk, dv = 9, 4, 3
    q, k, v, dO = rnd(1, T, 1, dk, seed=1), rnd(1, T, 1, dk, seed=2), rnd(1, T, 1, dv, seed=3), rnd(1, T, 1, dv, seed=4)
    g, S0, dS = -rnd(1, T, 1, seed=5).abs(), rnd(1, 1, dk, dv, seed=6), rnd(1, 1, dk, dv, seed=7)
    gq, gk, gv, gg, gS = ref.bwd(q, k, v, g, S0, None, dO, dS)
    tr = lambda S: S.transpose(-1, -2)  # noqa: E731
    fq, _ = ref.fwd(dO, v, k, g, tr(S0))
    assert torch.allclose(fq, gq, atol=1e-12)
    # reversed in time the decay between two tokens is the later one's: shifted by one
    r = lambda x: x.flip(1)  # noqa: E731
    gs = torch.cat([torch.zeros(1, 1, 1, dtype=torch.float64), r(g)[:, :-1]], 1)
    fk, _ = ref.fwd(r(v), r(dO), r(q), gs, tr(dS))
    fv, R = ref.fwd(r(k), r(q), r(dO), gs, dS)
    assert torch.allclose(r(fk), gk, atol=1e-12) and torch.allclose(r(fv), gv, atol=1e-12)
    assert torch.allclose(torch.exp(g[0, 0, 0]) * R, gS, atol=1e-12)
    _, S_T = ref.fwd(q, k, v, g, S0)
    d = (q * gq).sum(-1) - (k * gk).sum(-1)
    assert torch.allclose((S_T * dS).sum() + r(r(d).cumsum(1)), gg, atol=1e-12)


def test_reference_rotary():
    """A turn by pos * f keeps lengths, the inverse undoes it, and q.k depends on distance only."""
    f = [1.0, 0.1, 0.003]
    q, k = rnd(2, 1, 8, seed=1), rnd(2, 1, 8, seed=2)
    for layout in ("half", "interleaved"):
        for a, b in ((3, 7), (1003, 1007)):
            x = ref.rotary(q[:1], torch.tensor([a]), f, layout)
            y = ref.rotary(k[:1], torch.tensor([b]), f, layout)
            dot = float((x[..., :6] * y[..., :6]).sum())
            if a == 3:
                first = dot
            assert abs(dot - first) < 1e-10
            back = ref.rotary(x, torch.tensor([a]), f, layout, inverse=True)
            assert torch.allclose(back, q[:1], atol=1e-12)
        assert torch.equal(x[..., 6:], q[:1, :, 6:])


def fwd_call(lib, B=1, T=8, H=4, Hq=4, Hk=4, Hv=4, dk=64, dv=64, decay=0, io=0, n_seqs=0, cu=None,
             ptr=4096, ws=4096, nbytes=1 << 40, null=None, odd=None):
    p = {n: ptr for n in ("q", "k", "v", "g", "S0", "o", "S_T")}
    if null:
        p[null] = None
    if odd:
        p[odd] = ptr + 2
    return lib.ckda_linattn_fwd(p["q"], p["k"], p["v"], p["g"], p["S0"], cu, n_seqs, B, T, H, Hq, Hk,
                                Hv, dk, dv, decay, io, p["o"], p["S_T"], ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(null="q"), -1), (dict(null="k"), -1), (dict(null="v"), -1), (dict(null="g"), -1),
    (dict(dk=48), -2), (dict(dv=256), -2), (dict(H=0), -2), (dict(H=4, Hq=3), -2), (dict(Hk=0), -2),
    (dict(Hv=8), -2), (dict(B=-1), -2), (dict(T=-1), -2), (dict(B=70000, T=70000), -2),
    (dict(H=65536, Hq=1, Hk=1, Hv=1), -2), (dict(cu=4096, n_seqs=2, B=2), -2),
    (dict(cu=4096, n_seqs=-1), -2), (dict(cu=4096, n_seqs=0), -2),
    (dict(decay=2), -4), (dict(io=2), -4), (dict(odd="q"), -5), (dict(odd="S0"), -5),
    (dict(odd="g"), -5), (dict(odd="o"), -5), (dict(ws=None), -7), (dict(ws=4096 + 16), -7),
    (dict(nbytes=255), -7),
])
def test_fwd_refusals(lib, kw, code):
    assert fwd_call(lib, **kw) == code


def test_bwd_refusals(lib):
    def call(null=None, odd=None, nbytes=1 << 40, **kw):
        a = dict(B=1, T=8, H=4, Hq=4, Hk=2, Hv=1, dk=64, dv=64, decay=0, io=0)
        a.update(kw)
        p = {n: 4096 for n in ("q", "k", "v", "g", "S0", "dO", "dS_T", "dq", "dk", "dv", "dg", "dS0")}
        if null:
            p[null] = None
        if odd:
            p[odd] += 2
        return lib.ckda_linattn_bwd(p["q"], p["k"], p["v"], p["g"], p["S0"], None, 0, *a.values(), p["dO"],
                                    p["dS_T"], p["dq"], p["dk"], p["dv"], p["dg"], p["dS0"], 4096, nbytes, None)

    for n in ("q", "k", "v", "g", "dq", "dk", "dv", "dg"):
        assert call(null=n) == -1, n
    for n in ("q", "k", "v", "g", "S0", "dO", "dS_T", "dq", "dk", "dv", "dg", "dS0"):
        assert call(odd=n) == -5, n
    assert call(Hv=3) == -2 and call(dk=20) == -2 and call(io=3) == -4 and call(nbytes=1000) == -7


def test_decode_and_rotary_refusals(lib):
    def dec(null=None, odd=None, **kw):
        a = dict(B=1, H=4, Hq=4, Hk=2, Hv=1, dk=64, dv=64, decay=0, io=0)
        a.update(kw)
        p = {n: 4096 for n in ("q", "k", "v", "g", "S", "o")}
        if null:
            p[null] = None
        if odd:
            p[odd] += 2
        return lib.ckda_linattn_decode_step(p["q"], p["k"], p["v"], p["g"], p["S"], *a.values(), p["o"], None)

    assert all(dec(null=n) == -1 for n in ("q", "k", "v", "g", "S"))
    assert all(dec(odd=n) == -5 for n in ("q", "k", "v", "g", "S", "o"))
    assert dec(dk=8) == -2 and dec(Hq=3) == -2 and dec(decay=-1) == -4 and dec(io=7) == -4

    def rot(n=1, Hq=1, Hk=1, d=8, nf=4, layout=0, p64=0, io=0, null=None, odd=None):
        p = {x: 4096 for x in ("q", "k", "pos", "freqs", "qo", "ko")}
        if null:
            p[null] = None
        if odd:
            p[odd] += 2
        return lib.ckda_rotary(p["q"], p["k"], p["pos"], p["freqs"], n, Hq, Hk, d, nf, layout, p64, 1.0, 0,
                               io, p["qo"], p["ko"], None)

    assert all(rot(null=x) == -1 for x in ("q", "k", "pos", "freqs", "qo", "ko"))
    assert all(rot(odd=x) == -5 for x in ("q", "k", "pos", "freqs", "qo", "ko"))
    assert rot(nf=5) == -2 and rot(nf=-1) == -2 and rot(d=0) == -2 and rot(d=2048) == -2
    assert rot(n=-1) == -2 and rot(n=1 << 32) == -2 and rot(Hq=0) == -2 and rot(Hk=-1) == -2
    assert rot(Hq=65535) == -2 and rot(layout=2) == -4 and rot(io=2) == -4


def test_binding_refusals():
    q = torch.zeros(2, 5, 4, 64)
    k, v, g = torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 1, 32), torch.zeros(2, 5, 4)
    S = torch.zeros(2, 4, 64, 32)

    def bad(msg, **kw):
        a = dict(q=q, k=k, v=v, g=g)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            ops.linattn_fwd(**a)

    bad("must divide", k=torch.zeros(2, 5, 3, 64))
    bad("channels", k=torch.zeros(2, 5, 2, 32))
    bad("q's dtype", v=v.bfloat16())
    bad("float32 or bfloat16", q=q.half(), k=k.half(), v=v.half())
    bad("g must", g=g.bfloat16())
    bad("g must", g=torch.zeros(2, 4, 4))
    bad("k must", k=torch.zeros(2, 4, 2, 64))
    bad("S0 must", S0=torch.zeros(1, 4, 64, 32))
    bad("S_T must", S_T=S.bfloat16())
    bad("o must", o=torch.zeros(2, 5, 4, 64))
    bad("B == 1", cu_seqlens=torch.zeros(3, dtype=torch.int32))
    bad("int32", cu_seqlens=torch.zeros(3, dtype=torch.int64))
    bad("CUDA")
    with pytest.raises(ValueError, match="dO must"):
        ops.linattn_bwd(q, k, v, g, dO=torch.zeros(2, 5, 4, 64))
    with pytest.raises(ValueError, match="dS0 buffer"):
        ops.linattn_bwd(q, k, v, g, grads=(q, k, v, g, None))
    with pytest.raises(ValueError, match="dg must"):
        ops.linattn_bwd(q, k, v, g, grads=(q, k, v, g[..., :2], S))
    with pytest.raises(ValueError, match="S must"):
        ops.linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], S[:1])
    with pytest.raises(ValueError, match="one token|must be"):
        ops.linattn_decode_step(q, k, v, g, S)
    pos, f = torch.zeros(2, 5, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    for msg, kw in (("layout", dict(layout="both")), ("pos must", dict(pos=pos[:1])),
                    ("pos must", dict(pos=pos.float())), ("freqs must", dict(freqs=f.float())),
                    ("freqs must", dict(freqs=torch.zeros(33, dtype=torch.float64))),
                    ("k must", dict(k=k.bfloat16())), ("q_out must", dict(q_out=k)), ("CUDA", {})):
        a = dict(q=q, k=k, pos=pos, freqs=f)
        a.update(kw)
        with pytest.raises(ValueError, match=msg):
            ops.rotary(**a)
    with pytest.raises(ValueError, match="k_out without k"):
        ops.rotary(q, None, pos, f, k_out=k)


def test_rotary_freqs():
    f, s = ops.rotary_freqs(64, device="cpu")
    assert f.dtype == torch.float64 and f.numel() == 32 and s == 1.0
    assert f[0] == 1.0 and abs(float(f[16]) - 0.01) < 1e-15
    lin, _ = ops.rotary_freqs(64, scaling="linear", factor=8, device="cpu")
    assert torch.allclose(lin, f / 8, rtol=1e-14)
    base, _ = ops.rotary_freqs(64, scaling="base", factor=8, device="cpu")
    assert base[0] == 1.0 and abs(float(base[-1] / f[-1]) - 1 / 8) < 1e-12
    ramp, s = ops.rotary_freqs(64, scaling="ramp", factor=8, original_len=4096, device="cpu")
    assert ramp[0] == 1.0 and abs(float(ramp[-1] / f[-1]) - 1 / 8) < 1e-12
    assert s == pytest.approx(0.1 * math.log(8) + 1) and bool(((ramp <= f) & (ramp >= f / 8 * (1 - 1e-12))).all())
    for kw in (dict(dim=7), dict(dim=8, scaling="other"), dict(dim=8, scaling="linear", factor=0.5),
               dict(dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            ops.rotary_freqs(device="cpu", **kw)


def test_workspace_sizes(lib):
    """At least the header, growing with the call, and no smaller for gradients than forward."""
    w = lib.ckda_linattn_fwd_workspace_size
    for io in (0, 1):
        assert w(1, 0, 1, 16, 16, io, 0) >= 256
        assert w(1, 4096, 4, 64, 64, io, 0) >= w(1, 64, 4, 64, 64, io, 0) >= 256
        assert w(1, 4096, 4, 64, 64, io, 5) >= 256
        b = lib.ckda_linattn_bwd_workspace_size(1, 4096, 4, 4, 2, 1, 64, 64, 1, io, 0)
        assert b >= w(1, 4096, 4, 64, 64, io, 0)
    assert w(-1, 4, 4, 64, 64, 0, 0) == 256


def test_empty_calls_need_no_pointers(lib):
    """No token: the missing tensors are not an error, the workspace still is."""
    assert lib.ckda_linattn_fwd(None, None, None, None, None, None, 0, 2, 0, 4, 4, 4, 4, 64, 64, 0, 0, None,
                                None, None, 0, None) == -7
    assert lib.ckda_linattn_decode_step(None, None, None, None, None, 0, 4, 4, 4, 4, 65, 64, 0, 0, None,
                                        None) == -2
    assert ctypes.sizeof(ctypes.c_void_p) == 8


def test_shared_heads_up_to_the_most(tmp_path):
    """head_of(h, H, Hx), the head of a shared tensor that a kernel reads, is h * Hx // H for every size
    that the calls accept: from H = 46,342 on that product no longer fits 32 bits."""
    import os
    import subprocess

    src = os.path.join(lib_build.CSRC, "linattn.h")
    (tmp_path / "h.cc").write_text(f'''#include "{src}"
#include <cstdio>
int main() {{
  for (int H : {{1, 6, 46341, 46342, 50000, 65520, 65535}})
    for (int Hx = 1; Hx <= H; ++Hx) {{
      if (H % Hx) continue;
      for (int h = 0; h < H; ++h)
        if (ckda::head_of(h, H, Hx) != (long long)h * Hx / H) return std::printf("%d %d %d", h, H, Hx), 1;
    }}
  return 0;
}}''')
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(lib_build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", cuda, str(tmp_path / "h.cc"), "-o", str(tmp_path / "h")], check=True)
    r = subprocess.run([str(tmp_path / "h")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_longest_sequences(lib):
    """Up to 2^31 - 64 tokens: their segments are counted in 64 bits (the sum of a length and a segment's
    passes 32), so the workspace grows with the call; one token more is refused."""
    w, most = lib.ckda_linattn_fwd_workspace_size, 2**31 - 64
    for io in (0, 1):
        for n_seqs in (0, 1):
            half, full = w(1, 2**30, 1, 16, 16, io, n_seqs), w(1, most, 1, 16, 16, io, n_seqs)
            assert half <= full <= 2 * half + (1 << 20), (io, n_seqs, half, full)
    assert w(1, most, 1, 16, 16, 0, 0) >= (2**31 // 64) * 16 * 16 * 4
    assert fwd_call(lib, T=most + 1) == -2 and fwd_call(lib, T=most, nbytes=255) == -7


def test_rotary_freqs_on_the_first_device(monkeypatch):
    """device=0 is a device (and not the current one, whichever that is)."""
    asked = []
    monkeypatch.setattr(torch.Tensor, "to", lambda self, dev: asked.append(dev) or self)
    for dev in (0, 1, "cpu", None):
        ops.rotary_freqs(8, device=dev)
    assert asked == [0, 1, "cpu", "cuda"]
