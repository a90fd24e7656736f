"""Measured calls of linear attention with a decay for each head and of rotary positions.

Linear attention, per sequence and head, alpha_t = exp(g_t) with g_t <= 0:

    S_t = alpha_t S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t

as a whole prompt (``fwd``), as its gradients (``bwd``) and as one token on a resident state
(``decode``).  g is one log decay per token and head, or one per head.  Heads of q, k and v may
be shared: head h of H reads head h * Hx / H of a tensor that has Hx heads.  Rotary positions
turn channel pairs of q and k by position times frequency (``rotary``), and back for gradients.

``run`` computes the plain form (elementary torch operations, fp32, fp64 where exponents or
angles need it) or, with ``own``, calls the library.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_CHUNK = 64


# ------------------------------------------------------------------ cases
def _lin(name, op, dtype, B, T, H, Hq, Hk, Hv, dk, dv, fixed, state, lens_seed=0, n_short=0,
         short=0):
    """A linear attention case.  Packed when n_short > 0: n_short lengths up to ``short``, one
    sequence of T tokens and an empty one; else B sequences of T tokens.  ``state``: an initial
    state is given (and, backwards, a gradient of the final one)."""
    return dict(name=name, op=op, dtype=dtype, B=B, T=T, H=H, Hq=Hq, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                fixed=fixed, state=state, lens_seed=lens_seed, n_short=n_short, short=short)


def _rot(name, dtype, B, T, Hq, Hk, d, rot, layout, inverse, scaling, far):
    return dict(name=name, op="rotary", dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, d=d, rot=rot,
                layout=layout, inverse=inverse, scaling=scaling, far=far)


def listed():
    return [
        # a few dozen tokens in fp32, three heads: a call's fixed cost
        _lin("fwd_short_f32", "fwd", "f32", 2, 37, 3, 3, 3, 3, 64, 64, False, True),
        # a training batch's forward: four sequences, 16 heads of 128
        _lin("fwd_train", "fwd", "bf16", 4, 4096, 16, 16, 16, 16, 128, 128, False, False),
        # long sequences continued from a state, decays fixed per head
        _lin("fwd_long_fixed", "fwd", "bf16", 8, 8192, 16, 16, 16, 16, 128, 128, True, True),
        # prompts of many lengths packed together, one long and one empty, k and v shared by 4 heads
        _lin("fwd_packed_shared_kv", "fwd", "bf16", 1, 16384, 16, 16, 4, 4, 128, 128, False, True,
             lens_seed=1, n_short=12, short=4096),
        # the gradients of the training batch
        _lin("bwd_train", "bwd", "bf16", 4, 4096, 16, 16, 16, 16, 128, 128, False, False),
        # packed training sequences, q and k shared by 8 heads, smaller keys than values
        _lin("bwd_packed_shared_qk", "bwd", "bf16", 1, 2500, 16, 2, 2, 16, 64, 128, False, True,
             lens_seed=2, n_short=9, short=1500),
        # a small fp32 model's gradients, decays fixed per head, odd length
        _lin("bwd_f32_fixed", "bwd", "f32", 2, 515, 4, 4, 4, 4, 32, 64, True, True),
        # a full serving batch's next token
        _lin("decode_batch", "decode", "bf16", 256, 1, 32, 32, 32, 32, 128, 128, False, True),
        # one request's next token
        _lin("decode_one", "decode", "bf16", 1, 1, 16, 16, 16, 16, 128, 128, True, True),
        # a training batch's queries and keys
        _rot("rotary_train", "bf16", 4, 4096, 16, 16, 128, 128, "half", False, "none", False),
        # gradients of an odd fp32 batch, half of the head turned, shared keys
        _rot("rotary_grad_f32", "f32", 2, 2047, 16, 4, 128, 64, "interleaved", True, "none", False),
        # one token each of 64 requests far into their contexts, scaled frequencies
        _rot("rotary_decode_far", "bf16", 64, 1, 32, 8, 128, 128, "half", False, "ramp", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "decode", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rotary":
        d = rng.choice([32, 64, 128, 128])
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        B = _log_int(rng, 1, 256 if T == 1 else max(1, min(16, 32768 // T)))
        Hq = rng.randint(1, 32)
        Hk = rng.choice([h for h in range(1, Hq + 1) if Hq % h == 0])
        return dict(op="rotary", dtype=dtype, B=B, T=T, Hq=Hq, Hk=Hk, d=d,
                    rot=2 * rng.choice([d // 2, d // 4, rng.randint(1, d // 2)]),
                    layout=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "ramp"]), far=rng.random() < 0.5)
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64), (32, 32), (16, 64)])
    H = rng.randint(1, 16)
    div = [h for h in range(1, H + 1) if H % h == 0]
    Hq, Hk, Hv = rng.choice([(H, H, H), (H, rng.choice(div), None), (rng.choice(div), None, H)])[:3]
    Hv = Hk if Hv is None else Hv
    Hk = Hq if Hk is None else Hk
    fixed, state = rng.random() < 0.3, rng.random() < 0.6
    if op == "decode":
        return dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256), T=1, H=H, Hq=Hq, Hk=Hk, Hv=Hv,
                    dk=dk, dv=dv, fixed=fixed, state=True, lens_seed=0, n_short=0, short=0)
    most = 16384 if dtype == "f32" else 131072
    T = _log_int(rng, 1, 2048 if dtype == "f32" else 16384)
    n_short = rng.choice([0, rng.randint(1, 24)])
    B = 1 if n_short else _log_int(rng, 1, 8)
    while B * T * H > most and H * T > most // 4:
        T = max(1, T // 2 + 1)
    B = max(1, min(B, most // (T * H)))
    return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hq=Hq, Hk=Hk, Hv=Hv, dk=dk, dv=dv, fixed=fixed,
                state=state, lens_seed=rng.randint(1, 1 << 20), n_short=n_short,
                short=max(1, min(T // rng.randint(1, 4), most // (H * max(n_short, 1)))))


def _lengths(c):
    """Sequence lengths of a packed case (None: B rows of T tokens).  They belong to the case."""
    if not c["n_short"]:
        return None
    r = np.random.default_rng(c["lens_seed"])
    lens = [int(x) for x in r.integers(1, c["short"] + 1, size=c["n_short"])]
    at = len(lens) // 2
    return lens[:at] + [0] + lens[at:] + [c["T"]]


def _frequencies(c):
    """Radians per position of each channel pair (fp64) and the factor on the turned channels.
    linear: positions of an 8 times longer context pressed into the old range.  ramp: slow pairs
    pressed, fast ones kept, a linear ramp between, and the factor that goes with it."""
    n = c["rot"] // 2
    f = 10000.0 ** (-np.arange(n, dtype=np.float64) / n)
    scale = 1.0
    if c["scaling"] == "linear":
        f = f / 8.0
    elif c["scaling"] == "ramp":
        turns = 4096 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f / 32.0 * (1 - keep) + f * keep
        scale = 0.1 * math.log(32.0) + 1.0
    return f, scale


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = _DT[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["op"] == "rotary":
        B, T = c["B"], c["T"]
        top = 1_000_000 if c["far"] else 8192
        start = torch.randint(0, top, (B, 1), generator=gen, device=dev, dtype=torch.int32)
        pos = start + torch.arange(T, device=dev, dtype=torch.int32)
        f, scale = _frequencies(c)
        lead = (B, T) if T > 1 else (B,)   # a batch of prompts, or one token of each request
        return dict(case=c, q=normal(*lead, c["Hq"], c["d"]).to(dt),
                    k=normal(*lead, c["Hk"], c["d"]).to(dt), pos=pos.reshape(lead).contiguous(),
                    freqs=torch.from_numpy(f).to(dev), scale=scale)

    H, dk, dv = c["H"], c["dk"], c["dv"]
    lens = _lengths(c)
    if c["op"] == "decode":
        lead, N = (c["B"],), c["B"]
    elif lens is None:
        lead, N = (c["B"], c["T"]), c["B"]
    else:
        lead, N = (1, sum(lens)), len(lens)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    s = dict(case=c, lens=lens, q=unit(normal(*lead, c["Hq"], dk)), k=unit(normal(*lead, c["Hk"], dk)),
             v=normal(*lead, c["Hv"], dv).to(dt))
    if c["fixed"]:
        # slopes spread geometrically over the heads, moved a little by the seed
        h = torch.arange(1, H + 1, device=dev, dtype=torch.float32)
        s["g"] = -torch.exp2(-8.0 * h / H) * (1 + 0.1 * torch.rand(H, generator=gen, device=dev))
    else:
        s["g"] = torch.nn.functional.logsigmoid(4.0 + normal(*lead, H))
    s["S"] = 0.02 * normal(N, H, dk, dv) if c["state"] else None
    s["cu"] = None
    if lens is not None:
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)
    if c["op"] == "bwd":
        s["dO"] = normal(*lead, H, dv).to(dt)
        s["dS_T"] = 0.1 * normal(N, H, dk, dv) if c["state"] else None
    return s


# ------------------------------------------------------------------ the plain form
def _plain_linear(q, k, v, g, S0, lens):
    """o (fp32) and the final states of whole sequences, chunk by chunk side by side: scores
    within a chunk, the chunks' own states, and each chunk's incoming state as a weighted sum of
    the earlier ones'.  Differences of summed log decays are taken in fp64."""
    B, T = q.shape[:2]
    H = g.shape[-1]
    dk, dv, dev = q.shape[-1], v.shape[-1], q.device
    N = B if lens is None else len(lens)
    C = min(_CHUNK, max(1, T))
    if lens is None:
        blocks, nc = B, (T + C - 1) // C
        first = torch.arange(N, device=dev) * nc
        last = first + nc - 1
        in_seq = torch.arange(nc, device=dev).repeat(B)
        seq = torch.arange(B, device=dev).repeat_interleave(nc)
        start, length = torch.arange(B, device=dev) * T, torch.full((B,), T, device=dev)
    else:
        ln = np.asarray(lens, dtype=np.int64)
        per = (ln + C - 1) // C
        base = np.cumsum(per) - per
        blocks, nc = 1, int(per.sum())
        first = torch.from_numpy(base).to(dev)
        last = torch.from_numpy(np.maximum(base + per - 1, 0)).to(dev)
        seq = torch.from_numpy(np.repeat(np.arange(N), per)).to(dev)
        in_seq = torch.arange(nc, device=dev) - first[seq]
        start = torch.from_numpy(np.cumsum(ln) - ln).to(dev)
        length = torch.from_numpy(ln).to(dev)
    at = in_seq[:, None] * C + torch.arange(C, device=dev)
    valid = at < length[seq][:, None]                                  # [M, C]
    rows = torch.where(valid, start[seq][:, None] + at, 0)

    def chunks(x):                                                     # [M, H, C, d]
        x = x.reshape(B * T, *x.shape[2:])
        x = x.repeat_interleave(H // x.shape[1], dim=1)[rows]
        return torch.where(valid[:, :, None, None], x, 0.0).transpose(1, 2)

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    gd = g.double()
    gd = gd.expand(B * T, H) if g.dim() == 1 else gd.reshape(B * T, H)
    gc = torch.where(valid[:, :, None], gd[rows], 0.0).transpose(1, 2)   # [M, H, C]
    G = gc.cumsum(-1)
    total = G[..., -1]
    causal = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~causal, -math.inf).float().exp()
    o = ((qc @ kc.transpose(-1, -2)) * decay) @ vc
    local = (kc * (total[..., None] - G).float().exp()[..., None]).transpose(-1, -2) @ vc
    # states between chunks: [blocks, H, nc, nc] weights on the chunks' own states
    tot = total.reshape(blocks, nc, H).transpose(1, 2)
    upto = tot.cumsum(-1)
    before = upto - tot
    same = seq.reshape(blocks, nc)
    earlier = (same[:, :, None] == same[:, None, :]) & torch.ones(nc, nc, dtype=torch.bool, device=dev).tril(-1)
    W = (before[..., :, None] - upto[..., None, :]).masked_fill(~earlier[:, None], -math.inf).float().exp()
    loc = local.reshape(blocks, nc, H, dk * dv).transpose(1, 2)
    S_in = (W @ loc).transpose(1, 2).reshape(blocks * nc, H, dk, dv)
    if S0 is not None:
        bef = before.transpose(1, 2).reshape(blocks * nc, H)
        since = (bef - bef[first.clamp(max=max(blocks * nc - 1, 0))][seq]).float().exp()
        S_in = S_in + since[..., None, None] * S0[seq]
    o = o + (qc * G.float().exp()[..., None]) @ S_in
    S_out = total.float().exp()[..., None, None] * S_in + local
    ends = S_out[last]
    empty = (length == 0)[:, None, None, None]
    S_T = torch.where(empty, torch.zeros_like(ends) if S0 is None else S0, ends)
    out = o.transpose(1, 2)[valid].reshape(B, T, H, dv)
    return out, S_T


def _plain_rotary(x, pos, freqs, scale, layout, inverse):
    angle = pos.double()[..., None] * freqs
    cos = (angle.cos() * scale).float()[..., None, :]
    sin = (angle.sin() * (-scale if inverse else scale)).float()[..., None, :]
    n = freqs.numel()
    xf = x.float()
    if layout == "half":
        a, b = xf[..., :n], xf[..., n:2 * n]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = xf[..., 0:2 * n:2], xf[..., 1:2 * n:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([turned, xf[..., 2 * n:]], dim=-1).to(x.dtype)


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "rotary":
        return dict(zip("qk", (_plain_rotary(s[n], s["pos"], s["freqs"], s["scale"], c["layout"],
                                             c["inverse"]) for n in "qk")))
    q, k, v, g, dt = s["q"], s["k"], s["v"], s["g"], s["q"].dtype
    if c["op"] == "decode":
        H, S = c["H"], s["S"]
        qf, kf, vf = (x.float().repeat_interleave(H // x.shape[1], dim=1) for x in (q, k, v))
        S.mul_(g.exp().expand(c["B"], H)[..., None, None]).add_(kf[..., :, None] * vf[..., None, :])
        return {"o": (S * qf[..., :, None]).sum(-2).to(dt), "S": S}
    if c["op"] == "fwd":
        o, S_T = _plain_linear(q.float(), k.float(), v.float(), g, s["S"], s["lens"])
        return {"o": o.to(dt), "S_T": S_T}
    wrt = [x.float().detach().clone().requires_grad_() for x in (q, k, v, g)]
    S0 = s["S"].detach().clone().requires_grad_() if s["S"] is not None else None
    o, S_T = _plain_linear(*wrt, S0, s["lens"])
    loss = (o * s["dO"].float()).sum()
    if s["dS_T"] is not None:
        loss = loss + (S_T * s["dS_T"]).sum()
    grads = torch.autograd.grad(loss, wrt + ([S0] if S0 is not None else []))
    out = {"dq": grads[0].to(dt), "dk": grads[1].to(dt), "dv": grads[2].to(dt), "dg": grads[3]}
    if S0 is not None:
        out["dS0"] = grads[4]
    return out


def _own(s):
    from linear_rnn_ckda_b200 import ops

    c = s["case"]
    if c["op"] == "rotary":
        q, k = ops.rotary(s["q"], s["k"], s["pos"], s["freqs"], layout=c["layout"],
                          inverse=c["inverse"], scale=s["scale"])
        return {"q": q, "k": k}
    if c["op"] == "decode":
        o = ops.linattn_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"])
        return {"o": o, "S": s["S"]}
    if c["op"] == "fwd":
        o, S_T = ops.linattn_fwd(s["q"], s["k"], s["v"], s["g"], S0=s["S"], cu_seqlens=s["cu"])
        return {"o": o, "S_T": S_T}
    dq, dk, dv, dg, dS0 = ops.linattn_bwd(s["q"], s["k"], s["v"], s["g"], S0=s["S"],
                                          cu_seqlens=s["cu"], dO=s["dO"], dS_T=s["dS_T"],
                                          want_dS0=s["S"] is not None)
    out = {"dq": dq, "dk": dk, "dv": dv, "dg": dg}
    if dS0 is not None:
        out["dS0"] = dS0
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "rotary":
        n = c["B"] * c["T"]
        x = n * (c["Hq"] + c["Hk"])
        return {"bytes": 2 * x * c["d"] * es + 4 * n + 4 * c["rot"], "flops": 3 * x * c["rot"]}
    lens = _lengths(c)
    tok = sum(lens) if lens is not None else c["B"] * c["T"]
    N = len(lens) if lens is not None else c["B"]
    H, dk, dv = c["H"], c["dk"], c["dv"]
    ins = tok * ((c["Hq"] + c["Hk"]) * dk + c["Hv"] * dv) * es
    o = tok * H * dv * es
    g = (H if c["fixed"] else tok * H) * 4
    state = N * H * dk * dv * 4
    if c["op"] == "decode":
        return {"bytes": ins + o + g + 2 * state, "flops": 5 * tok * H * dk * dv}
    if c["op"] == "fwd":
        return {"bytes": ins + o + g + state * (2 if c["state"] else 1), "flops": 4 * tok * H * dk * dv}
    return {"bytes": 2 * ins + o + 2 * g + state * (3 if c["state"] else 0),
            "flops": 10 * tok * H * dk * dv}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Token by token in fp64."""
    c, s = case, prepare(case, seed)
    if c["op"] == "rotary":
        th = s["pos"].double()[..., None, None] * s["freqs"]
        turn = torch.polar(torch.full_like(th, s["scale"]), -th if c["inverse"] else th)
        n, out = s["freqs"].numel(), {}
        for name in "qk":
            x = s[name].double()
            y = x.clone()
            i = torch.arange(n, device=x.device)
            i, j = (i, i + n) if c["layout"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., i].contiguous(), x[..., j].contiguous()) * turn
            y[..., i], y[..., j] = z.real, z.imag
            out[name] = y
        return out
    H, dk, dv = c["H"], c["dk"], c["dv"]
    q, k, v, g = (s[n].double() for n in ("q", "k", "v", "g"))
    if c["op"] == "decode":
        head = lambda x: torch.stack([x[:, h * x.shape[1] // H] for h in range(H)], 1)  # noqa: E731
        S = g.exp().expand(c["B"], H)[..., None, None] * s["S"].double()
        S = S + torch.einsum("bhi,bhj->bhij", head(k), head(v))
        return {"o": torch.einsum("bhij,bhi->bhj", S, head(q)), "S": S}
    lens = s["lens"] or [c["T"]] * c["B"]
    N, Tm, dev = len(lens), max(lens), q.device
    off = [0] + [int(x) for x in np.cumsum(lens)]
    alone = {"n": N * H, "q": (c["Hq"], dk), "k": (c["Hk"], dk), "v": (c["Hv"], dv), "dO": (H, dv)}

    def spread(x, hx, d):
        """[Tm, N * H, d]: sequences side by side, rows past a sequence's end zero."""
        x = x.reshape(-1, hx, d)
        y = torch.zeros(Tm, N, H, d, dtype=torch.float64, device=dev)
        for n in range(N):
            y[:lens[n], n] = x[off[n]:off[n + 1], [h * hx // H for h in range(H)]]
        return y.reshape(Tm, N * H, d)

    qs, ks, vs = (spread(x, *alone[n]) for n, x in (("q", q), ("k", k), ("v", v)))
    gt = spread(g.expand(off[-1], H).reshape(-1, H) if g.dim() == 1 else g, H, 1)   # 0 past the end
    al = gt.exp()[..., None]
    zero = torch.zeros(N * H, dk, dv, dtype=torch.float64, device=dev)
    S = zero.clone() if s["S"] is None else s["S"].double().reshape(N * H, dk, dv).clone()
    back = c["op"] == "bwd"
    if back:
        dO = spread(s["dO"].double(), *alone["dO"])
    got = torch.empty(Tm, N * H, dk if back else dv, dtype=torch.float64, device=dev)
    for t in range(Tm):
        S.mul_(al[t]).baddbmm_(ks[t, :, :, None], vs[t, :, None, :])
        got[t] = torch.bmm(S, dO[t, :, :, None])[..., 0] if back else torch.bmm(qs[t, :, None, :], S)[:, 0]

    def packed(y):
        y = y.reshape(Tm, N, H, -1)
        return torch.cat([y[:lens[n], n] for n in range(N)], 0)

    if not back:
        return {"o": packed(got).reshape(*s["q"].shape[:2], H, dv), "S_T": S.reshape(N, H, dk, dv)}
    R = zero.clone() if s["dS_T"] is None else s["dS_T"].double().reshape(N * H, dk, dv).clone()
    slope = (S * R).sum((-1, -2))
    dks, dvs = torch.empty_like(ks), torch.empty_like(vs)
    for t in range(Tm - 1, -1, -1):
        R.baddbmm_(qs[t, :, :, None], dO[t, :, None, :])
        dks[t] = torch.bmm(R, vs[t, :, :, None])[..., 0]
        dvs[t] = torch.bmm(ks[t, :, None, :], R)[:, 0]
        R.mul_(al[t])
    dG = (got * qs).sum(-1) - (dks * ks).sum(-1)
    dg = packed((dG.flip(0).cumsum(0).flip(0) + slope)[..., None])[..., 0]

    def shared(y, hx):
        y = packed(y)
        return y.reshape(y.shape[0], hx, H // hx, -1).sum(2)

    out = {"dq": shared(got, c["Hq"]).reshape(s["q"].shape), "dk": shared(dks, c["Hk"]).reshape(s["k"].shape),
           "dv": shared(dvs, c["Hv"]).reshape(s["v"].shape),
           "dg": dg.sum(0) if g.dim() == 1 else dg.reshape(s["g"].shape)}
    if s["S"] is not None:
        out["dS0"] = R.reshape(N, H, dk, dv)
    return out
