"""Linear attention with a decay for each head on the GPU against the float64 token loop.

Tolerances (relative Frobenius error, assert_close): fp32 results hold the library's fp32 bar,
1e-5 (sums of a few hundred products, each rounded by 2^-24, stay below 1e-6), and dg, a
difference of sums, the backward's 1e-4.  bf16 outputs are rounded once (at most 2^-8 of a
value, in the mean square at most 2^-8 / sqrt 3) and may read a state and scores rounded
likewise, whose errors add in squares: sqrt 2 * 2^-8 / sqrt 3 = 3.2e-3 < 2^-8."""
import math

import numpy as np
import pytest
import torch

import linattn_ref as ref
from helpers import assert_close, f64

pytestmark = pytest.mark.gpu
TOL = {torch.float32: 1e-5, torch.bfloat16: 2.0 ** -8}
TOL_DG = 1e-4
F32, BF = torch.float32, torch.bfloat16


def make(B, T, H, Hq, Hk, Hv, dk, dv, dtype, fixed=False, N=None, state=True, seed=0, gate=4.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    N = B if N is None else N
    t = dict(q=unit(r(B, T, Hq, dk)).to(dtype), k=unit(r(B, T, Hk, dk)).to(dtype), v=r(B, T, Hv, dv).to(dtype))
    if fixed:
        t["g"] = -torch.exp2(-8.0 * torch.arange(1, H + 1) / H).float()
    else:
        t["g"] = torch.nn.functional.logsigmoid(gate + r(B, T, H)).float()
    t["S0"] = (0.1 * r(N, H, dk, dv)).float() if state else None
    return t, (r(B, T, H, dv).to(dtype), r(N, H, dk, dv).float() if state else None)


def cuda(t):
    return {n: None if x is None else x.cuda() for n, x in t.items()}


def normal(x):
    """Values below fp32's smallest normal number, 2^-126, as 0: there fp32 is spaced by 2^-149, so
    no relative tolerance holds (a value of 5e-45 is off by up to 2^-150 = 7e-46, 14 % of it)."""
    x = np.array(x, dtype=np.float64)
    x[np.abs(x) < 2.0 ** -126] = 0.0
    return x


def offsets(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)


def check_fwd(ops, t, cu=None):
    d = cuda(t)
    o, S = ops.linattn_fwd(**d, cu_seqlens=None if cu is None else cu.cuda())
    ro, rS = ref.fwd(**t, cu=cu)
    dt = t["q"].dtype
    assert o.dtype == dt and S.dtype == F32
    assert_close(f64(o), ro.numpy(), TOL[dt], "o", bf16_out=dt == BF)
    assert_close(normal(f64(S)), normal(rS.numpy()), TOL[F32], "S_T")
    return o, S


def check_bwd(ops, t, dO, dS, cu=None):
    d = cuda(t)
    got = ops.linattn_bwd(**d, cu_seqlens=None if cu is None else cu.cuda(),
                          dO=None if dO is None else dO.cuda(), dS_T=None if dS is None else dS.cuda())
    want = ref.bwd(**t, cu=cu, dO=dO, dS_T=dS)
    dt = t["q"].dtype
    for name, x, y in zip(("dq", "dk", "dv", "dg", "dS0"), got, want):
        low = name in ("dq", "dk", "dv")
        assert x.dtype == (dt if low else F32) and bool(torch.isfinite(x).all()), name
        y = y.detach().numpy()
        if name == "dg":
            assert_close(f64(x).reshape(-1, x.shape[-1]), y.reshape(-1, y.shape[-1]), TOL_DG, name)
        else:
            x, y = (f64(x), y) if low else (normal(f64(x)), normal(y))
            assert_close(x, y, TOL[dt] if low else TOL[F32], name, bf16_out=low and dt == BF)


HEADS = [(3, 3, 3, 3), (4, 4, 2, 2), (4, 1, 1, 4), (6, 2, 3, 1)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 200])
def test_fwd_lengths(cuda_lib, T, dtype):
    check_fwd(cuda_lib, make(2, T, 2, 2, 2, 2, 128, 128, dtype, seed=T)[0])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 128), (128, 32), (64, 64), (16, 128), (128, 64)])
def test_dims(cuda_lib, dk, dv, dtype):
    t, (dO, dS) = make(1, 130, 2, 2, 2, 2, dk, dv, dtype, seed=dk + dv)
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("H,Hq,Hk,Hv", HEADS)
@pytest.mark.parametrize("fixed", [False, True])
def test_shared_heads(cuda_lib, H, Hq, Hk, Hv, fixed, dtype):
    t, (dO, dS) = make(2, 70, H, Hq, Hk, Hv, 32, 64, dtype, fixed=fixed, seed=H + Hq)
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1, 0, 64, 65, 0, 63, 7], [0, 0, 300], [0], [0, 1, 0], [128, 128]])
def test_packed(cuda_lib, lens, dtype):
    t, (dO, dS) = make(1, sum(lens), 2, 2, 2, 2, 64, 128, dtype, N=len(lens), seed=len(lens))
    cu = offsets(lens)
    check_fwd(cuda_lib, t, cu)
    check_bwd(cuda_lib, t, dO, dS, cu)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T", [1, 64, 129])
def test_bwd_lengths(cuda_lib, T, dtype):
    t, (dO, dS) = make(2, T, 2, 2, 2, 2, 128, 128, dtype, seed=T)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_missing_parts(cuda_lib, dtype):
    """No S0; no dO; no dS_T; nothing wanted but one output."""
    t, (dO, _) = make(1, 100, 2, 2, 2, 2, 64, 64, dtype, state=False)
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, None)
    t, (dO, dS) = make(1, 100, 2, 2, 2, 2, 64, 64, dtype)
    check_bwd(cuda_lib, t, None, dS)
    check_bwd(cuda_lib, t, dO, None)
    d = cuda(t)
    o, S = cuda_lib.linattn_fwd(**d)
    o1, none = cuda_lib.linattn_fwd(**d, want_state=False)
    none2, S1 = cuda_lib.linattn_fwd(**d, want_o=False)
    assert none is None and none2 is None and torch.equal(o, o1) and torch.equal(S, S1)
    got = cuda_lib.linattn_bwd(**d, dO=dO.cuda(), want_dS0=False)
    assert got[4] is None


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_sequences(cuda_lib, dtype):
    """Long enough to be split over many SMs; few and many heads, slow decays."""
    for B, T, H in ((1, 4000, 1), (2, 1500, 3)):
        t, (dO, dS) = make(B, T, H, H, H, H, 64, 64, dtype, seed=T, gate=7.0)
        check_fwd(cuda_lib, t)
        check_bwd(cuda_lib, t, dO, dS)
    lens = [2000, 0, 37, 900]
    t, (dO, dS) = make(1, sum(lens), 2, 2, 1, 1, 128, 128, dtype, N=4, seed=9, gate=6.0)
    check_fwd(cuda_lib, t, offsets(lens))
    check_bwd(cuda_lib, t, dO, dS, offsets(lens))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_extreme_decays(cuda_lib, dtype):
    """Resets (-inf), decays that underflow within a chunk, exact ones (0), in one batch."""
    t, (dO, dS) = make(1, 200, 3, 3, 3, 3, 64, 64, dtype, seed=3)
    g = t["g"]
    g[0, :, 0] = 0.0
    g[0, 10::37, 1] = -math.inf
    g[0, :, 2] = -60.0
    g[0, 100:110, 2] = -1e30
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("gap", [0, 40])
def test_chunks_that_decay_fast_but_not_at_once(cuda_lib, gap, dtype):
    """64 tokens lose 2^-138, 32 of them 2^-69: a chunk's weights leave fp32's range, a half's do
    not.  (`gap` tokens without decay first, so that such chunks stand beside ordinary ones.)"""
    t, (dO, dS) = make(2, 150 + gap, 2, 1, 2, 2, 64, 128, dtype, seed=gap)
    t["g"] = torch.full_like(t["g"], -1.5)
    t["g"][:, :gap] = 0.0
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[40], [700], [3, 0, 640, 64]])
def test_states_in_place(cuda_lib, lens, dtype):
    """S_T over S0 and dS0 over dS_T give the bits that separate buffers give."""
    T, N = sum(lens), len(lens)
    t, (dO, dS) = make(1, T, 4, 2, 4, 4, 64, 128, dtype, N=N, seed=T)
    d, cu = cuda(t), offsets(lens).cuda()
    dO, dS = dO.cuda(), dS.cuda()
    o, S_T = cuda_lib.linattn_fwd(**d, cu_seqlens=cu)
    grads = cuda_lib.linattn_bwd(**d, cu_seqlens=cu, dO=dO, dS_T=dS)
    over = d["S0"].clone()
    o2, S2 = cuda_lib.linattn_fwd(**{**d, "S0": over}, cu_seqlens=cu, S_T=over)
    assert S2 is over and torch.equal(S2, S_T) and torch.equal(o2, o)
    room = [torch.empty_like(d[n]) for n in ("q", "k", "v", "g")] + [dS.clone()]
    again = cuda_lib.linattn_bwd(**d, cu_seqlens=cu, dO=dO, dS_T=room[4], grads=room)
    assert all(torch.equal(x, y) for x, y in zip(again, grads))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_two_calls_at_once(cuda_lib, dtype):
    """Forward and backward calls in flight on two streams give the bits that they give alone."""
    sets, alone = [], []
    for seed in (1, 2):
        t, (dO, dS) = make(1, 700, 8, 8, 4, 8, 128, 128, dtype, seed=seed)
        sets.append((cuda(t), dO.cuda(), dS.cuda()))
    run = lambda x: (*cuda_lib.linattn_fwd(**x[0]), *cuda_lib.linattn_bwd(**x[0], dO=x[1], dS_T=x[2]))  # noqa: E731
    for x in sets:
        alone.append(run(x))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, x in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(run(x))
        torch.cuda.synchronize()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_large_sums_of_decays(cuda_lib):
    """A chunk that starts with a thousandfold underflow and then decays slowly: the weights among
    the later tokens keep fp32 accuracy although their summed decays are large."""
    t, (dO, dS) = make(1, 128, 1, 1, 1, 1, 64, 64, F32, seed=4)
    t["g"][0, :, 0] = -0.001
    t["g"][0, 0:30, 0] = -99.7
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_values_stay_in_their_sequence(cuda_lib, dtype):
    """NaN and infinity in one sequence (all its inputs) leave the neighbours' results as they are."""
    lens = [30, 70, 100, 5]
    t, (dO, dS) = make(1, sum(lens), 2, 2, 2, 2, 64, 64, dtype, N=4, seed=5)
    cu = offsets(lens).cuda()
    d = cuda(t)
    clean = cuda_lib.linattn_fwd(**d, cu_seqlens=cu)
    clean_b = cuda_lib.linattn_bwd(**d, cu_seqlens=cu, dO=dO.cuda(), dS_T=dS.cuda())
    for val in (math.nan, math.inf):
        e = {n: x.clone() for n, x in d.items()}
        do = dO.cuda().clone()
        for n in ("q", "k", "v"):
            e[n][0, 30:100] = val
        e["g"][0, 30:100] = math.nan
        do[0, 30:100] = val
        o, S = cuda_lib.linattn_fwd(**e, cu_seqlens=cu)
        keep = torch.ones(sum(lens), dtype=torch.bool)
        keep[30:100] = False
        assert torch.equal(o[0, keep], clean[0][0, keep])
        assert torch.equal(S[[0, 2, 3]], clean[1][[0, 2, 3]])
        got = cuda_lib.linattn_bwd(**e, cu_seqlens=cu, dO=do, dS_T=dS.cuda())
        for x, y in zip(got[:4], clean_b[:4]):
            assert torch.equal(x[0, keep], y[0, keep])
        assert torch.equal(got[4][[0, 2, 3]], clean_b[4][[0, 2, 3]])


def test_bad_offsets_write_nothing(cuda_lib):
    t, _ = make(1, 100, 2, 2, 2, 2, 64, 64, BF, N=3)
    d = cuda(t)
    good = torch.tensor([0, 20, 60, 100], dtype=torch.int32, device="cuda")
    n = cuda_lib.linattn_fwd_workspace_size(1, 100, 2, 64, 64, BF, 3)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for bad in ([0, 60, 20, 100], [0, 20, 60, 90], [1, 20, 60, 100], [0, 20, 400, 100], [0, -5, 60, 100]):
        o = torch.full((1, 100, 2, 64), 7.0, dtype=BF, device="cuda")
        S = torch.full((3, 2, 64, 64), 7.0, device="cuda")
        cuda_lib.linattn_fwd(**d, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), o=o, S_T=S,
                             workspace=ws)
        assert cuda_lib.workspace_status(ws) == -6
        assert bool((o == 7).all()) and bool((S == 7).all())
    cuda_lib.linattn_fwd(**d, cu_seqlens=good, o=o, S_T=S, workspace=ws)
    assert cuda_lib.workspace_status(ws) == 0
    ro, _ = ref.fwd(**t, cu=good.cpu())
    assert_close(f64(o), ro.numpy(), TOL[BF], "o", bf16_out=True)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_in_parts_and_tokens(cuda_lib, dtype):
    """A prompt, the same in two parts through the state (S_T in S0's place), and token by token."""
    t, _ = make(2, 150, 4, 4, 2, 2, 64, 64, dtype, seed=6)
    d = cuda(t)
    o, S = cuda_lib.linattn_fwd(**d)
    cut = lambda a, b: {n: d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")}  # noqa: E731
    St = d["S0"].clone()
    oa, _ = cuda_lib.linattn_fwd(**cut(0, 71), S0=St, S_T=St)
    ob, _ = cuda_lib.linattn_fwd(**cut(71, 150), S0=St, S_T=St)
    ro, rS = ref.fwd(**t)
    assert_close(f64(torch.cat([oa, ob], 1)), ro.numpy(), TOL[dtype], "parts", bf16_out=dtype == BF)
    assert_close(f64(St), rS.numpy(), TOL[F32], "S of parts")
    St = d["S0"].clone()
    steps = [cuda_lib.linattn_decode_step(*(d[n][:, i].contiguous() for n in ("q", "k", "v", "g")), St)
             for i in range(150)]
    assert_close(f64(torch.stack(steps, 1)), ro.numpy(), TOL[dtype], "tokens", bf16_out=dtype == BF)
    assert_close(f64(St), rS.numpy(), TOL[F32], "S of tokens")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("B,H,Hq,Hk,Hv,dk,dv,fixed", [
    (1, 1, 1, 1, 1, 128, 128, False), (3, 6, 2, 3, 6, 64, 16, True), (5, 4, 4, 1, 1, 16, 128, False),
    (2, 2, 2, 2, 2, 32, 32, True), (64, 32, 32, 8, 8, 128, 64, False)])
def test_decode(cuda_lib, B, H, Hq, Hk, Hv, dk, dv, fixed, dtype):
    t, _ = make(B, 1, H, Hq, Hk, Hv, dk, dv, dtype, fixed=fixed, seed=B)
    d = cuda(t)
    g = d["g"] if fixed else d["g"][:, 0].contiguous()
    args = [d[n][:, 0].contiguous() for n in ("q", "k", "v")] + [g]
    S, S1 = d["S0"].clone(), d["S0"].clone()
    o = cuda_lib.linattn_decode_step(*args, S)
    assert cuda_lib.linattn_decode_step(*args, S1, want_o=False) is None
    ro, rS = ref.fwd(**t)
    assert_close(f64(o), ro[:, 0].numpy(), TOL[dtype], "o", bf16_out=dtype == BF)
    assert_close(f64(S), rS.numpy(), TOL[F32], "S")
    assert torch.equal(S, S1)


def test_decode_unaligned_and_empty(cuda_lib):
    """q, k, v, o that start at an odd element; B = 0."""
    t, _ = make(3, 1, 2, 2, 2, 2, 64, 64, BF, seed=8)
    d = cuda(t)
    odd = lambda x: torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape)  # noqa: E731
    args = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g")]
    Sa, Sb = d["S0"].clone(), d["S0"].clone()
    o = cuda_lib.linattn_decode_step(*args, Sa)
    ob = cuda_lib.linattn_decode_step(*(odd(x) for x in args), Sb, o=odd(torch.zeros_like(o)))
    assert torch.equal(o, ob) and torch.equal(Sa, Sb)
    e = cuda_lib.linattn_decode_step(*(x[:0] for x in args), Sa[:0])
    assert e.shape == (0, 2, 64)


def test_empty_calls(cuda_lib):
    for B, T in ((0, 5), (2, 0)):
        t, (dO, dS) = make(B, T, 2, 2, 2, 2, 64, 64, BF, fixed=True, seed=1)
        d = cuda(t)
        o, S = cuda_lib.linattn_fwd(**d)
        assert o.shape == (B, T, 2, 64) and torch.equal(S, d["S0"])
        got = cuda_lib.linattn_bwd(**d, dO=dO.cuda(), dS_T=dS.cuda())
        assert torch.equal(got[4], dS.cuda()) and bool((got[3] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_same_bits_again_and_in_graphs(cuda_lib, dtype):
    """Repeats, another stream, and two captured graphs replayed in turn give the same bits."""
    t, (dO, dS) = make(2, 333, 4, 4, 2, 2, 64, 128, dtype, seed=7)
    d, dO, dS = cuda(t), dO.cuda(), dS.cuda()

    def call():
        return [*cuda_lib.linattn_fwd(**d), *cuda_lib.linattn_bwd(**d, dO=dO, dS_T=dS)]

    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = call()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call()
        graphs.append((g, out))
    for _ in range(2):
        for g, out in graphs:
            for x in out:
                x.zero_()
            g.replay()
    torch.cuda.synchronize()
    for x, y, a, b in zip(first, other, graphs[0][1], graphs[1][1]):
        assert torch.equal(x, y) and torch.equal(x, a) and torch.equal(x, b)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_rotary_then_attention(cuda_lib, dtype):
    """Rotary positions, linear attention and its gradients back through the turn, as a layer
    runs them; then one more token of each sequence from the state."""
    B, T, H, Hk, d_ = 2, 90, 4, 2, 64
    t, (dO, dS) = make(B, T + 1, H, H, Hk, Hk, d_, d_, dtype, seed=11)
    dS = dS * 0.1
    d = cuda(t)
    pos = (torch.arange(T + 1, dtype=torch.int32) + torch.tensor([[5], [100000]], dtype=torch.int32))
    freqs, scale = cuda_lib.rotary_freqs(48, scaling="ramp", factor=4.0)
    part = lambda n, a, b: d[n][:, a:b].contiguous()  # noqa: E731
    qr, kr = cuda_lib.rotary(part("q", 0, T), part("k", 0, T), pos[:, :T].contiguous().cuda(), freqs, scale=scale)
    o, S = cuda_lib.linattn_fwd(qr, kr, part("v", 0, T), part("g", 0, T), S0=d["S0"])
    dq, dk, dv, dg, dS0 = cuda_lib.linattn_bwd(qr, kr, part("v", 0, T), part("g", 0, T), S0=d["S0"],
                                               dO=dO[:, :T].contiguous().cuda(), dS_T=dS.cuda())
    dq, dk = cuda_lib.rotary(dq, dk, pos[:, :T].contiguous().cuda(), freqs, scale=scale, inverse=True)
    # the same in float64, fed the kernel's own rounded q and k
    want = ref.bwd(qr.cpu(), kr.cpu(), t["v"][:, :T], t["g"][:, :T], t["S0"], None, dO[:, :T], dS)
    wq, wk = (ref.rotary(x.detach(), pos[:, :T], freqs.cpu(), "half", inverse=True, scale=scale) for x in want[:2])
    ro, rS = ref.fwd(qr, kr, t["v"][:, :T], t["g"][:, :T], t["S0"])
    b = dtype == BF
    assert_close(f64(o), ro.numpy(), TOL[dtype], "o", bf16_out=b)
    # (a second rounding on the way back: bf16 errors add in squares, sqrt 3 / sqrt 3 * 2^-8)
    for x, y, n in ((dq, wq, "dq"), (dk, wk, "dk")):
        assert_close(f64(x), y.numpy(), 2 * TOL[dtype], n, bf16_out=b)
    tok = pos[:, T].contiguous().cuda()
    q1, k1 = cuda_lib.rotary(d["q"][:, T].contiguous(), d["k"][:, T].contiguous(), tok, freqs, scale=scale)
    o1 = cuda_lib.linattn_decode_step(q1, k1, d["v"][:, T].contiguous(), d["g"][:, T].contiguous(), S)
    r1, _ = ref.fwd(q1[:, None], k1[:, None], t["v"][:, T:], t["g"][:, T:], rS)
    assert_close(f64(o1), r1[:, 0].numpy(), TOL[dtype], "o of the next token", bf16_out=b)


def decay_gradient(q, k, v, g, dO):
    """dg of sum(dO o) in float64 on the GPU, token by token: g's share of S_t = e^g S_{t-1} + k v^T is
    e^{g_t} <S_{t-1}, R_t>, R_t the gradient of S_t; <S_T, 0> plus the suffix sums of q.dq - k.dk."""
    q, k, v, g, dO = (x.double() for x in (q, k, v, g, dO))
    B, T, H, dk = q.shape
    S = torch.zeros(B, H, dk, v.shape[-1], dtype=torch.float64, device=q.device)
    R, dots = S.clone(), torch.zeros(B, T, H, dtype=torch.float64, device=q.device)
    a = g.exp()[..., None, None]
    for t in range(T):
        S.mul_(a[:, t]).add_(k[:, t, :, :, None] * v[:, t, :, None, :])
        dots[:, t] += ((S * dO[:, t, :, None, :]).sum(-1) * q[:, t]).sum(-1)
    for t in range(T - 1, -1, -1):
        R.add_(q[:, t, :, :, None] * dO[:, t, :, None, :])
        dots[:, t] -= ((R * v[:, t, :, None, :]).sum(-1) * k[:, t]).sum(-1)
        R.mul_(a[:, t])
    return dots.flip(1).cumsum(1).flip(1)


def test_decay_gradients_of_long_sequences(cuda_lib):
    """bf16 inputs, a training batch whose sequences stay in few segments.  dg is a sum of q.dq - k.dk
    over up to a segment's tokens.  The tensor cores truncate an accumulator at each addition, by
    2^-24 of its value in the mean over all mantissas (half a step of 2^-23, times ln 2 and more): with
    one addition per 16 of 128 channels and 64 tokens at full size, 12 x 2^-24 x ln 2 = 5e-7 of dq and
    of dk, and so of dg, at most the sum of both: 1e-6.  (An addition for each of three terms would
    be three times as many.)"""
    t, (dO, _) = make(2, 3000, 26, 26, 26, 26, 128, 128, BF, state=False, seed=21)
    d, dO = cuda(t), dO.cuda()
    got = cuda_lib.linattn_bwd(**d, dO=dO, want_dS0=False)[3].double()
    want = decay_gradient(d["q"], d["k"], d["v"], d["g"], dO)
    assert float((got - want).norm() / want.norm()) <= 1e-6


@pytest.mark.parametrize("decay", [None, -1.5, -6.0])
def test_bf16_results_are_rounded_once(cuda_lib, decay):
    """bf16 outputs and gradients against the float64 ones rounded to bf16.  The kernel's operands (state
    and scores) keep 17 bits and more: each at most 2^-18 off, so a result is at most about 2^-17 off
    before it is rounded, and only values that lie that near a border between two bf16 values (steps of at
    least 2^-8 of the value), 2 x 2^-17 / 2^-8 = 2^-8 of them, may fall on its other side, by a step of
    at most 2^-7: sqrt(2^-8) x 2^-7 = 2^-11 in the mean square.  (Operands of 8 bits: 2.6e-3.)"""
    t, (dO, dS) = make(2, 300, 4, 4, 2, 4, 128, 64, BF, seed=31)
    if decay is not None:
        t["g"] = torch.full_like(t["g"], decay)
    d = cuda(t)
    o, _ = cuda_lib.linattn_fwd(**d)
    grads = cuda_lib.linattn_bwd(**d, dO=dO.cuda(), dS_T=dS.cuda())[:3]
    want = [ref.fwd(**t)[0]] + [x.detach() for x in ref.bwd(**t, dO=dO, dS_T=dS)[:3]]
    for x, y, name in zip((o, *grads), want, ("o", "dq", "dk", "dv")):
        once = y.to(BF).double()
        assert float((x.double().cpu() - once).norm() / once.norm()) <= 2.0 ** -11, name


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_heads(cuda_lib, dtype):
    """50,000 heads (their product with a tensor's heads passes 32 bits), own and shared ones: one
    token, a prompt and its gradients."""
    H = 50_000
    t, (dO, dS) = make(1, 3, H, H, H // 2, H, 16, 16, dtype, seed=41)
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO, dS)
    d = cuda(t)
    S = d["S0"].clone()
    o = cuda_lib.linattn_decode_step(*(d[n][:, 0].contiguous() for n in ("q", "k", "v", "g")), S)
    ro, rS = ref.fwd(**{n: x if n == "S0" else x[:, :1] for n, x in t.items()})
    assert_close(f64(o), ro[:, 0].numpy(), TOL[dtype], "o", bf16_out=dtype == BF)
    assert_close(f64(S), rS.numpy(), TOL[F32], "S")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("decay", [-0.85, -1.05, -1.5, -3.0])
@pytest.mark.parametrize("log2", [20, -12])
def test_large_and_small_values_with_fast_decays(cuda_lib, log2, decay, dtype):
    """Values of a million and of a four-thousandth where a chunk of 64 tokens loses 2^-78 to 2^-277: no
    factor on the way may leave fp32's range while the results (2^60 and 2^-36) are far inside it."""
    t, (dO, dS) = make(2, 150, 2, 2, 1, 2, 64, 128, dtype, seed=log2 + 50)
    f = 2.0 ** log2
    for n in ("q", "k", "v"):
        t[n] = t[n] * f
    t["S0"] = t["S0"] * f * f
    t["g"] = torch.full_like(t["g"], decay)
    check_fwd(cuda_lib, t)
    check_bwd(cuda_lib, t, dO * f, dS * f * f)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("fixed", [False, True])
@pytest.mark.parametrize("T", [60, 200, 1500])
def test_nan_decay_shows(cuda_lib, T, fixed, dtype):
    """A NaN log decay makes NaN of everything it reaches (as in a decode step), in its own head and
    sequence only; chunks of 64 tokens before it (after it for dk and dv) keep their bits."""
    t, (dO, dS) = make(2, T, 3, 3, 3, 3, 64, 64, dtype, fixed=fixed, seed=T)
    at = T // 2
    d, dO, dS = cuda(t), dO.cuda(), dS.cuda()
    run = lambda: (*cuda_lib.linattn_fwd(**d), *cuda_lib.linattn_bwd(**d, dO=dO, dS_T=dS))  # noqa: E731
    clean = run()
    d["g"] = d["g"].clone()
    d["g"][(1,) if fixed else (0, at, 1)] = math.nan
    got = run()
    lo, hi = (0, T) if fixed else (at // 64 * 64, min(T, at // 64 * 64 + 64))
    for n, x, y in zip(("o", "S_T", "dq", "dk", "dv", "dg", "dS0"), got, clean):
        if n == "dg" and fixed:
            assert bool(torch.isnan(x[1])) and torch.equal(x[[0, 2]], y[[0, 2]])
            continue
        heads = (lambda z: z) if n in ("S_T", "dS0") else (lambda z: z.transpose(1, 2))  # noqa: E731
        x, y = heads(x), heads(y)                    # [B, H, ..]
        assert torch.equal(x[:, [0, 2]], y[:, [0, 2]]), n
        bad, ok = x[0, 1], y[0, 1]
        if not fixed:
            assert torch.equal(x[1, 1], y[1, 1]), n
        if n in ("S_T", "dS0", "dg"):
            assert bool(torch.isnan(bad).all()), n
        elif n in ("o", "dq"):
            assert bool(torch.isnan(bad[0 if fixed else at:]).all()) and torch.equal(bad[:lo], ok[:lo]), n
        else:
            assert bool(torch.isnan(bad[:T if fixed else at]).all()) and torch.equal(bad[hi:], ok[hi:]), n


@pytest.mark.parametrize("dtype", [F32, BF])
def test_decay_gradients_where_nothing_is_left(cuda_lib, dtype):
    """A token whose decay leaves nothing of the state has gradient 0 itself, and so has a sequence's
    first token without S0; the others of each head keep their accuracy on the head's own scale."""
    t, (dO, _) = make(2, 700, 3, 3, 3, 3, 64, 64, dtype, state=False, seed=61)
    g = t["g"]
    g[0, 10::37, 1] = -math.inf
    g[0, 100:110, 2] = -1e30
    g[1, 20::50, 0] = -88.0
    got = cuda_lib.linattn_bwd(**cuda(t), dO=dO.cuda())[3].double().cpu()
    want = ref.bwd(**t, dO=dO)[3].detach()
    assert bool((got[g < -87.4] == 0).all()) and bool((got[:, 0] == 0).all())
    for h in range(3):
        assert float((got[:, :, h] - want[:, :, h]).norm() / want[:, :, h].norm()) <= TOL_DG, h


def test_decay_gradients_of_one_long_segment(cuda_lib):
    """bf16, so many sequences that each stays whole.  Each of the 12 additions at full size that make
    up an element of dq truncates by up to 2^-23, 2^-23 / sqrt 12 in the mean square, and q . dq sums
    independent elements: 2^-23 of q . dq, sqrt 2 of that with k . dk.  A sum of n such errors, tied at both
    ends, is sqrt(n / 6) of one in the mean square over its tokens (tied at one end sqrt(n / 2))."""
    n = 6000
    t, (dO, _) = make(4, n, 40, 40, 40, 40, 128, 128, BF, state=False, seed=71)
    d, dO = cuda(t), dO.cuda()
    got = cuda_lib.linattn_bwd(**d, dO=dO, want_dS0=False)
    want = decay_gradient(d["q"], d["k"], d["v"], d["g"], dO)
    rho = float((got[0].float() * d["q"].float()).sum(-1).pow(2).mean().sqrt())
    size = float(want.pow(2).mean().sqrt())
    tol = math.sqrt(2 * n / 6) * 2.0 ** -23 * rho / size + 5e-7
    assert float((got[3].double() - want).pow(2).mean().sqrt()) / size <= tol


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("chunk", [0, 2])
def test_a_wait_that_runs_out(cuda_lib, chunk, packed):
    """A role that waits for nothing (test hook, 0.2 ms): every unit that reaches that chunk ends, the
    status word says so, and the next calls in the same workspace give the bits they gave before."""
    # (forty heads and more than that in sequences of 500 tokens: their segments have three chunks and more)
    B, T, lens = (1, 2000, [700, 0, 30, 1270]) if packed else (4, 500, None)
    N = len(lens) if packed else B
    t, (dO, dS) = make(B, T, 40, 40, 20, 40, 64, 128, BF, N=N, seed=81)
    d, dO, dS = cuda(t), dO.cuda(), dS.cuda()
    cu = offsets(lens).cuda() if packed else None
    n = max(cuda_lib.linattn_bwd_workspace_size(B, T, 40, 40, 20, 40, 64, 128, 0, BF, N if packed else 0),
            cuda_lib.linattn_fwd_workspace_size(B, T, 40, 64, 128, BF, N if packed else 0))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def fwd():
        return cuda_lib.linattn_fwd(**d, cu_seqlens=cu, workspace=ws)

    def bwd():
        return cuda_lib.linattn_bwd(**d, cu_seqlens=cu, dO=dO, dS_T=dS, workspace=ws)

    for call in (fwd, bwd):
        want = call()
        assert cuda_lib.workspace_status(ws) == 0
        try:
            cuda_lib.debug_wait_injection(chunk, 200_000)
            call()
            assert cuda_lib.workspace_status(ws) == -8      # CKDA_ERR_TIMEOUT
        finally:
            cuda_lib.debug_wait_injection(-1, 0)
        again = call()
        assert cuda_lib.workspace_status(ws) == 0
        assert all(torch.equal(x, y) for x, y in zip(want, again))
