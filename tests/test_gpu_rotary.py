"""Rotary positions on the GPU against the float64 definition.  fp32: the angle's fraction of a
turn is rounded once (2^-25 of half a turn, 1e-7 radians) and products a few times by 2^-24, far
below 1e-6; bf16 outputs are that, rounded once (2^-8 of the value, checked element by element)."""
import numpy as np
import pytest
import torch

import linattn_ref as ref

pytestmark = pytest.mark.gpu
F32, BF = torch.float32, torch.bfloat16


def close(x, y, what):
    """Element by element: 1e-6 of the largest value a pair can reach, and half a step in bf16."""
    x, y = x.detach().double().cpu(), y.double()
    tol = 1e-6 * float(y.abs().max().clamp(min=1e-30)) + (0 if what == F32 else 2.0 ** -8 * y.abs())
    assert bool(((x - y).abs() <= tol).all()), float((x - y).abs().max())


def rnd(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,n", [(128, 64), (128, 32), (64, 5), (6, 3), (33, 16), (20, 0), (8, 4), (256, 128), (24, 4)])
def test_layouts_and_sizes(cuda_lib, d, n, layout, dtype):
    q, k = rnd(2, 7, 3, d, seed=1, dtype=dtype), rnd(2, 7, 2, d, seed=2, dtype=dtype)
    pos = torch.arange(14, dtype=torch.int32).reshape(2, 7) * 37
    f = torch.tensor(10000.0 ** (-np.arange(n) / max(n, 1)), dtype=torch.float64)
    for inverse, scale in ((False, 1.0), (True, 1.25)):
        a, b = cuda_lib.rotary(q.cuda(), k.cuda(), pos.cuda(), f.cuda(), layout=layout, inverse=inverse, scale=scale)
        for x, y in ((q, a), (k, b)):
            close(y, ref.rotary(x, pos, f, layout, inverse, scale), dtype)
            assert torch.equal(y[..., 2 * n:].cpu(), x[..., 2 * n:])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_far_positions(cuda_lib, dtype):
    """Positions of many turns, negative ones, and int64 past 32 bits: angles against exact
    arithmetic (Python integers on the fp64 frequencies' exact fractions of a turn)."""
    from fractions import Fraction
    import math

    f = torch.tensor([1.0, 0.37, 1e-3, 2.5, 0.0], dtype=torch.float64)
    pos = torch.tensor([0, 1, 999_999, 2**31 - 1, -5, -123_456, 2**33 + 7, 2**40], dtype=torch.int64)
    q = rnd(len(pos), 1, 10, seed=3, dtype=dtype)
    got, none = cuda_lib.rotary(q.cuda(), None, pos.cuda(), f.cuda())
    assert none is None
    # 2 pi to 30 digits; angle modulo a turn exactly.  The kernel's frequency in turns is an fp64
    # product, off by 2^-53 of itself, so the angle by 2^-53 pos f: allowed for beside the fp32 part.
    turn = Fraction(628318530717958647692528676655901, 10**32)
    want = q.double().clone()
    slack = torch.zeros(len(pos), dtype=torch.float64)
    for t, p in enumerate(pos.tolist()):
        for i, fi in enumerate(f.tolist()):
            x = Fraction(fi) * p
            a = float(x - turn * (x // turn))
            c, s = math.cos(a), math.sin(a)
            u, w = q[t, 0, i].double(), q[t, 0, i + 5].double()
            want[t, 0, i], want[t, 0, i + 5] = u * c - w * s, w * c + u * s
            slack[t] = max(float(slack[t]), abs(p * fi) * 2.0 ** -52)
    err = (got.double().cpu() - want).abs()
    tol = (1e-6 + slack[:, None, None]) * 4.0 + (2.0 ** -8 * want.abs() if dtype == BF else 0)
    assert bool((err <= tol).all()), err.max()
    small = pos[:6].to(torch.int32)
    again, _ = cuda_lib.rotary(q[:6].cuda(), None, small.cuda(), f.cuda())
    assert torch.equal(again, got[:6])


def test_in_place_unaligned_empty_and_single(cuda_lib):
    f = torch.tensor(10000.0 ** (-np.arange(32) / 32), dtype=torch.float64, device="cuda")
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    for dtype in (F32, BF):
        q, k = rnd(50, 4, 96, seed=4, dtype=dtype).cuda(), rnd(50, 1, 96, seed=5, dtype=dtype).cuda()
        a, b = cuda_lib.rotary(q, k, pos, f)
        q1, k1 = q.clone(), k.clone()
        r = cuda_lib.rotary(q1, k1, pos, f, q_out=q1, k_out=k1)
        assert r[0] is q1 and torch.equal(q1, a) and torch.equal(k1, b)
        odd = torch.cat([q.new_zeros(1), q.flatten()])[1:].view(q.shape)
        assert torch.equal(cuda_lib.rotary(odd, k, pos, f)[0], a)
        one = cuda_lib.rotary(q[7:8], k[7:8], pos[7:8], f)
        assert torch.equal(one[0], a[7:8]) and torch.equal(one[1], b[7:8])
        e = cuda_lib.rotary(q[:0], k[:0], pos[:0], f)
        assert e[0].shape == (0, 4, 96)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_tokens(cuda_lib, dtype):
    """Several tokens per block and a last block that is not full; every token against its own call."""
    n = 3001
    q, k = rnd(n, 5, 64, seed=6, dtype=dtype).cuda(), rnd(n, 5, 64, seed=7, dtype=dtype).cuda()
    f, _ = cuda_lib.rotary_freqs(32)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") * 11
    a, b = cuda_lib.rotary(q, k, pos, f, layout="interleaved")
    for lo in (0, 1000, n - 200):
        for x, y in ((q, a), (k, b)):
            close(y[lo:lo + 200], ref.rotary(x[lo:lo + 200], pos[lo:lo + 200], f.cpu(), "interleaved"), dtype)
    back, _ = cuda_lib.rotary(a.float(), None, pos, f, layout="interleaved", inverse=True)
    assert float((back - q.float()).abs().max()) < (1e-5 if dtype == F32 else 2.0 ** -7 * float(q.float().abs().max()) * 1.5)


def test_angles_at_any_position(cuda_lib):
    """fp32, positions up to 2^44 and frequencies of many turns, none and negative ones: the angle is off
    by 2^-63 of a turn per position, 2 pi 2^-63 |pos| radians, and by fp32's rounding of its fraction of a
    turn and of the results (the 1e-6 of the other tests, of values up to 4)."""
    from fractions import Fraction
    import math

    f = torch.tensor([1.0, 0.37, 1e-3, 2.5, -0.7, 1e-9, 1000.1, 3e15], dtype=torch.float64)
    pos = torch.tensor([1, 999_999, -2**31, 2**33 + 7, -2**40 - 1, 2**42 + 3, 2**44 - 5], dtype=torch.int64)
    q = rnd(len(pos), 1, 16, seed=13, dtype=F32).clamp(-4, 4)
    got, _ = cuda_lib.rotary(q.cuda(), None, pos.cuda(), f.cuda())
    # 2 pi to 60 digits
    turn = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10**60)
    for t, p in enumerate(pos.tolist()):
        for i, fi in enumerate(f.tolist()):
            x = Fraction(fi) * p
            a = float(x - turn * (x // turn))
            c, s = math.cos(a), math.sin(a)
            u, w = q[t, 0, i].double(), q[t, 0, i + 8].double()
            tol = 4.0 * (1e-6 + abs(p) * 2.0 * math.pi * 2.0 ** -63)
            assert abs(float(got[t, 0, i]) - float(u * c - w * s)) <= tol, (p, fi)
            assert abs(float(got[t, 0, i + 8]) - float(w * c + u * s)) <= tol, (p, fi)
