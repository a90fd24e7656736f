"""Python binding of ``libckda.so`` (the C ABI in ``include/ckda.h``).

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the recurrence runs in the library's kernels.
There is no CPU fallback: if the library is missing or the tensors are not on
a CUDA device, these functions raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libckda.so")
_lock = threading.Lock()
_lib = None

CKDA_F32 = 0
CKDA_BF16 = 1
# flags OR-ed into signed_gate (include/ckda.h)
GATE_PER_HEAD = 16   # one gate logit per token and head: a is [B,T,H] ([B,H] for decode)
QK_L2NORM = 32       # q and k are L2-normalised inside the kernels
DELTA_PRODUCT2 = 64  # two keys, values, strengths per token: k [B,T,2,H,dk], v [B,T,2,H,dv], b [B,T,2,H]
# how linear attention's log decays are given, and rotary channel pairs
DECAY_PER_TOKEN, DECAY_PER_HEAD = 0, 1
ROTARY_LAYOUTS = {"half": 0, "interleaved": 1}
_DT = {torch.float32: CKDA_F32, torch.bfloat16: CKDA_BF16}
_TORCH_DT = {CKDA_F32: torch.float32, CKDA_BF16: torch.bfloat16}

_vp = ctypes.c_void_p
_i = ctypes.c_int

# name -> (restype, argtypes), mirroring include/ckda.h
SIGNATURES = {
    "ckda_chunk_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _i, _i, _vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ckda_chunk_fwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i, _i]),
    "ckda_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp]),
    "ckda_chunk_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                            _vp]),
    "ckda_chunk_bwd_workspace_size": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "ckda_chunk_fwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i,
                                    _i, _i, _i, _vp, _vp, _vp]),
    "ckda_linattn_fwd": (_i, [_vp] * 6 + [_i] * 11 + [_vp, _vp, _vp, ctypes.c_size_t, _vp]),
    "ckda_linattn_fwd_workspace_size": (ctypes.c_size_t, [_i] * 7),
    "ckda_linattn_bwd": (_i, [_vp] * 6 + [_i] * 11 + [_vp] * 8 + [ctypes.c_size_t, _vp]),
    "ckda_linattn_bwd_workspace_size": (ctypes.c_size_t, [_i] * 11),
    "ckda_linattn_decode_step": (_i, [_vp] * 5 + [_i] * 9 + [_vp, _vp]),
    "ckda_rotary": (_i, [_vp] * 4 + [ctypes.c_longlong] + [_i] * 6 + [ctypes.c_float, _i, _i, _vp,
                                                                      _vp, _vp]),
    "ckda_workspace_status": (_i, [_vp, ctypes.POINTER(_i), _vp]),
    "ckda_noalloc_status": (_i, [ctypes.POINTER(_i), _vp]),
    "ckda_debug_wait_injection": (None, [_i, ctypes.c_ulonglong]),
    "ckda_debug_segment_split": (None, [_i, _i]),
    "ckda_debug_segment_choice": (_i, [ctypes.POINTER(ctypes.c_int32), _i, _i, _i,
                                      ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
    "ckda_status_string": (ctypes.c_char_p, [_i]),
    "ckda_version": (_i, []),
}


class CkdaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {status_string(code)} (code {code})")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def load():
    """Loads ``libckda.so`` (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is missing: build it with `python -m linear_rnn_ckda_b200.build` "
                    "(there is no CPU fallback)")
            lib = ctypes.CDLL(_LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().ckda_status_string(int(code)).decode()


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _same_device(ref: torch.Tensor, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != ref.device:
            raise ValueError(f"{name} is on {t.device}, q on {ref.device}")


def check_prefill_args(q, k, v, a, b, S0=None, cu_seqlens=None, o=None, S_T=None,
                       o_dtype=None, signed_gate: int = 0):
    """Shapes, dtypes and devices that ``ckda_chunk_fwd`` relies on but cannot see (it receives
    bare pointers, so a short or mistyped buffer would be read or written past its end).
    Raises ValueError; returns (N, dv).  The offsets inside ``cu_seqlens`` are checked on the
    device (the workspace status word), not here."""
    _need(q.dim() == 4, f"q must be [B,T,H,dk], got {tuple(q.shape)}")
    _need(q.dtype in _DT, f"q must be float32 or bfloat16, got {q.dtype}")
    B, T, H, dk = q.shape
    p2 = bool(signed_gate & DELTA_PRODUCT2)
    lead = (B, T, 2, H) if p2 else (B, T, H)   # rows of k, v, b (two per token for DeltaProduct2)
    _need(tuple(k.shape) == lead + (dk,) and k.dtype == q.dtype,
          f"k must be {lead + (dk,)} in q's dtype, got {tuple(k.shape)}, {k.dtype}")
    a_shape = (B, T, H) if signed_gate & GATE_PER_HEAD else tuple(q.shape)
    _need(tuple(a.shape) == a_shape and a.dtype == q.dtype,
          f"a must be {a_shape} in q's dtype, got {tuple(a.shape)}, {a.dtype}")
    _need(v.dim() == len(lead) + 1 and tuple(v.shape[:-1]) == lead and v.dtype == q.dtype,
          f"v must be {lead + ('dv',)} in q's dtype, got {tuple(v.shape)}, {v.dtype}")
    dv = v.shape[-1]
    _need(tuple(b.shape) == lead and b.dtype == torch.float32,
          f"b must be {lead} float32, got {tuple(b.shape)}, {b.dtype}")
    N = B
    if cu_seqlens is not None:
        _need(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1 and cu_seqlens.dtype == torch.int32,
              "cu_seqlens must be a 1-D int32 tensor of N+1 offsets")
        _need(B == 1, "packed sequences (cu_seqlens) need B == 1")
        N = cu_seqlens.numel() - 1
    for name, t in (("S0", S0), ("S_T", S_T)):
        _need(t is None or (t.shape == (N, H, dk, dv) and t.dtype == torch.float32),
              f"{name} must be [N,H,dk,dv] = {(N, H, dk, dv)} float32")
    od = q.dtype if o_dtype is None else o_dtype
    _need(od in _DT, f"o_dtype must be float32 or bfloat16, got {od}")
    _need(o is None or (o.shape == (B, T, H, dv) and o.dtype == od),
          f"o must be [B,T,H,dv] = {(B, T, H, dv)} in {od}")
    _same_device(q, k=k, v=v, a=a, b=b, S0=S0, cu_seqlens=cu_seqlens, o=o, S_T=S_T)
    return N, dv


def check_decode_args(q, k, v, a, b, S, o=None, o_dtype=None, signed_gate: int = 0):
    """The same checks for ``ckda_decode_step``: q, k, a [B,H,dk]; v [B,H,dv] in q's dtype;
    b [B,H] float32; S [B,H,dk,dv] float32; o [B,H,dv] in the output dtype."""
    _need(q.dim() == 3, f"q must be [B,H,dk], got {tuple(q.shape)}")
    _need(q.dtype in _DT, f"q must be float32 or bfloat16, got {q.dtype}")
    B, H, dk = q.shape
    lead = (B, 2, H) if signed_gate & DELTA_PRODUCT2 else (B, H)
    _need(tuple(k.shape) == lead + (dk,) and k.dtype == q.dtype,
          f"k must be {lead + (dk,)} in q's dtype, got {tuple(k.shape)}, {k.dtype}")
    a_shape = (B, H) if signed_gate & GATE_PER_HEAD else tuple(q.shape)
    _need(tuple(a.shape) == a_shape and a.dtype == q.dtype,
          f"a must be {a_shape} in q's dtype, got {tuple(a.shape)}, {a.dtype}")
    _need(v.dim() == len(lead) + 1 and tuple(v.shape[:-1]) == lead and v.dtype == q.dtype,
          f"v must be {lead + ('dv',)} in q's dtype, got {tuple(v.shape)}, {v.dtype}")
    dv = v.shape[-1]
    _need(tuple(b.shape) == lead and b.dtype == torch.float32,
          f"b must be {lead} float32, got {tuple(b.shape)}, {b.dtype}")
    _need(S.shape == (B, H, dk, dv) and S.dtype == torch.float32,
          f"S must be [B,H,dk,dv] = {(B, H, dk, dv)} float32")
    od = q.dtype if o_dtype is None else o_dtype
    _need(od in _DT, f"o_dtype must be float32 or bfloat16, got {od}")
    _need(o is None or (o.shape == (B, H, dv) and o.dtype == od),
          f"o must be [B,H,dv] = {(B, H, dv)} in {od}")
    _same_device(q, k=k, v=v, a=a, b=b, S=S, o=o)
    return dv


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def workspace_size(B, T, H, dk, dv, chunk, n_seqs=0) -> int:
    return int(load().ckda_chunk_fwd_workspace_size(B, T, H, dk, dv, chunk, n_seqs))


def new_workspace(B, T, H, dk, dv, chunk, n_seqs=0, device=None) -> torch.Tensor:
    n = workspace_size(B, T, H, dk, dv, chunk, n_seqs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def chunk_fwd(q, k, v, a, b, S0=None, cu_seqlens=None, chunk: int = 64, signed_gate: int = 1,
              o_dtype=None, o=None, S_T=None, workspace=None, want_o: bool = True,
              want_state: bool = True):
    """Chunkwise forward.  Returns (o, S_T) (either may be None when not wanted).

    q, k, a: [B,T,H,dk]; v: [B,T,H,dv] (fp32 or bf16, same dtype); b: [B,T,H] fp32;
    S0: [N,H,dk,dv] fp32 or None; cu_seqlens: int32 CUDA tensor [N+1] or None.
    """
    lib = load()
    N, dv = check_prefill_args(q, k, v, a, b, S0, cu_seqlens, o, S_T, o_dtype, signed_gate)
    B, T, H, dk = q.shape
    io = _DT[q.dtype]
    od = io if o_dtype is None else _DT[o_dtype]
    dev = q.device
    if want_o and o is None:
        o = torch.empty((B, T, H, dv), dtype=_TORCH_DT[od], device=dev)
    if want_state and S_T is None:
        S_T = torch.empty((N, H, dk, dv), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = new_workspace(B, T, H, dk, dv, chunk, N if cu_seqlens is not None else 0, dev)
    _need(workspace.device == dev, f"workspace is on {workspace.device}, q on {dev}")
    rc = lib.ckda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(S0),
                            _ptr(cu_seqlens), N if cu_seqlens is not None else 0, B, T, H, dk, dv,
                            chunk, signed_gate, io, od, _ptr(o if want_o else None),
                            _ptr(S_T if want_state else None), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(dev))
    if rc != 0:
        raise CkdaError("ckda_chunk_fwd", rc)
    return (o if want_o else None), (S_T if want_state else None)


def bwd_workspace_size(B, T, H, dk, dv, n_seqs=0) -> int:
    return int(load().ckda_chunk_bwd_workspace_size(B, T, H, dk, dv, n_seqs))


def chunk_bwd(q, k, v, a, b, S0=None, cu_seqlens=None, dO=None, dS_T=None,
              signed_gate: int = 1, want_dS0: bool = True, workspace=None, grads=None):
    """Backward of ``chunk_fwd``: gradients of sum(dO * o) + sum(dS_T * S_T).

    Returns (dq, dk, dv, da, db, dS0) as float32 tensors with the shapes of q, k, v, a, b and
    S0's [N,H,dk,dv] (dS0 None when not wanted).  dO: [B,T,H,dv] float32 or bfloat16, or None
    (zero); dS_T: [N,H,dk,dv] float32 or None (zero).  ``grads`` may supply the six output
    tensors."""
    lib = load()
    N, dv = check_prefill_args(q, k, v, a, b, S0, cu_seqlens, signed_gate=signed_gate)
    B, T, H, dk = q.shape
    dev = q.device
    _need(dO is None or (dO.shape == (B, T, H, dv) and dO.dtype in _DT),
          f"dO must be [B,T,H,dv] = {(B, T, H, dv)} float32 or bfloat16")
    _need(dS_T is None or (dS_T.shape == (N, H, dk, dv) and dS_T.dtype == torch.float32),
          f"dS_T must be [N,H,dk,dv] = {(N, H, dk, dv)} float32")
    _same_device(q, dO=dO, dS_T=dS_T)
    if grads is None:
        f32 = dict(dtype=torch.float32, device=dev)
        grads = (torch.empty((B, T, H, dk), **f32), torch.empty((B, T, H, dk), **f32),
                 torch.empty((B, T, H, dv), **f32), torch.empty(tuple(a.shape), **f32),
                 torch.empty((B, T, H), **f32),
                 torch.empty((N, H, dk, dv), **f32) if want_dS0 else None)
    gq, gk, gv, ga, gb, gS0 = grads
    for name, t, shape in (("dq", gq, (B, T, H, dk)), ("dk", gk, (B, T, H, dk)),
                           ("dv", gv, (B, T, H, dv)), ("da", ga, tuple(a.shape)),
                           ("db", gb, (B, T, H)), ("dS0", gS0, (N, H, dk, dv))):
        _need(t is None or (tuple(t.shape) == shape and t.dtype == torch.float32),
              f"{name} must be {shape} float32")
    _need(gS0 is not None or not want_dS0, "dS0 buffer missing")
    n = bwd_workspace_size(B, T, H, dk, dv, N if cu_seqlens is not None else 0)
    if workspace is None:
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    rc = lib.ckda_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(S0), _ptr(cu_seqlens),
                            N if cu_seqlens is not None else 0, B, T, H, dk, dv, signed_gate,
                            _DT[q.dtype], _ptr(dO), _DT[dO.dtype] if dO is not None else CKDA_F32,
                            _ptr(dS_T), _ptr(gq), _ptr(gk), _ptr(gv), _ptr(ga), _ptr(gb),
                            _ptr(gS0), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(dev))
    if rc != 0:
        raise CkdaError("ckda_chunk_bwd", rc)
    return gq, gk, gv, ga, gb, gS0


def decode_step(q, k, v, a, b, S, signed_gate: int = 1, o_dtype=None, o=None, want_o=True):
    """One decode step; S [B,H,dk,dv] fp32 is updated in place.  Returns o [B,H,dv]."""
    lib = load()
    dv = check_decode_args(q, k, v, a, b, S, o, o_dtype, signed_gate)
    B, H, dk = q.shape
    io = _DT[q.dtype]
    od = io if o_dtype is None else _DT[o_dtype]
    if want_o and o is None:
        o = torch.empty((B, H, dv), dtype=_TORCH_DT[od], device=q.device)
    rc = lib.ckda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(S), B, H, dk, dv,
                              signed_gate, io, od, _ptr(o if want_o else None), _stream(q.device))
    if rc != 0:
        raise CkdaError("ckda_decode_step", rc)
    return o if want_o else None


def noalloc_status(device=None) -> int:
    """Device status word of the last ``ckda_chunk_fwd_noalloc`` call on the current device
    (synchronises the current stream)."""
    st = ctypes.c_int(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    rc = load().ckda_noalloc_status(ctypes.byref(st), _stream(dev))
    if rc != 0:
        raise CkdaError("ckda_noalloc_status", rc)
    return st.value


def debug_wait_injection(chunk_index: int, wait_ns: int = 0) -> None:
    """Test hook: see ``ckda_debug_wait_injection`` in ``include/ckda.h`` (-1 switches it off)."""
    load().ckda_debug_wait_injection(int(chunk_index), int(wait_ns))


def debug_segment_choice(lengths, H: int, sm_count: int = 148):
    """Test hook: see ``ckda_debug_segment_choice`` in ``include/ckda.h``.  Returns
    (sequences cut, [segments of each])."""
    n = len(lengths)
    arr = (ctypes.c_int32 * max(n, 1))(*[int(x) for x in lengths])
    k = ctypes.c_int(0)
    m = (ctypes.c_int * 2)()
    rc = load().ckda_debug_segment_choice(arr, n, int(H), int(sm_count), ctypes.byref(k), m)
    if rc != 0:
        raise CkdaError("ckda_debug_segment_choice", rc)
    return k.value, [m[i] for i in range(k.value)]


def debug_segment_split(n_split: int, n_segments: int) -> None:
    """Test hook: see ``ckda_debug_segment_split`` in ``include/ckda.h`` (0, 0 switches it off)."""
    load().ckda_debug_segment_split(int(n_split), int(n_segments))


def workspace_status(workspace: torch.Tensor) -> int:
    """Device status word of the last chunk_fwd that used ``workspace`` (synchronises)."""
    st = ctypes.c_int(0)
    rc = load().ckda_workspace_status(_ptr(workspace), ctypes.byref(st), _stream(workspace.device))
    if rc != 0:
        raise CkdaError("ckda_workspace_status", rc)
    return st.value


# ------------------------------------------------------------------ linear attention
# These calls are short (a token of a small batch takes microseconds on the device), so their checks
# build no message and no tuple unless one fails.
def _lin_heads(g, lead, named):
    """(H, decay code, [heads of each tensor]) of linear attention tensors [*lead, Hx, d]."""
    gs, n = g.shape, len(lead)
    fixed = len(gs) == 1
    if g.dtype != torch.float32 or not (fixed or gs[:-1] == lead):
        raise ValueError(f"g must be {tuple(lead) + ('H',)} or [H] float32, got {tuple(gs)}, {g.dtype}")
    H, heads = gs[-1], []
    if H < 1:
        raise ValueError("g has no heads")
    for name, t in named:
        s = t.shape
        if len(s) != n + 2 or s[:n] != lead:
            raise ValueError(f"{name} must be {tuple(lead) + ('heads', 'channels')}, got {tuple(s)}")
        x = s[n]
        if x < 1 or H % x:
            raise ValueError(f"{name} has {x} heads, which must divide g's {H}")
        heads.append(x)
    return H, (DECAY_PER_HEAD if fixed else DECAY_PER_TOKEN), heads


def _lin_types(q, k, v):
    if q.dtype not in _DT:
        raise ValueError(f"q must be float32 or bfloat16, got {q.dtype}")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError(f"k and v must be in q's dtype {q.dtype}, got {k.dtype}, {v.dtype}")
    if k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q has {q.shape[-1]} channels, k {k.shape[-1]}")


def _lin_out(name, t, shape, dtype):
    """A given tensor's shape and dtype (None passes)."""
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)}, {t.dtype}")


def check_linattn_args(q, k, v, g, S0=None, cu_seqlens=None):
    """Shapes and dtypes that ``ckda_linattn_fwd`` and ``ckda_linattn_bwd`` cannot see.  Raises
    ValueError; returns (N, H, decay code, (Hq, Hk, Hv))."""
    if q.dim() != 4:
        raise ValueError(f"q must be [B,T,Hq,dk], got {tuple(q.shape)}")
    lead = q.shape[:2]
    H, decay, heads = _lin_heads(g, lead, (("q", q), ("k", k), ("v", v)))
    _lin_types(q, k, v)
    N = lead[0]
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or cu_seqlens.dtype != torch.int32:
            raise ValueError("cu_seqlens must be a 1-D int32 tensor of N+1 offsets")
        if lead[0] != 1:
            raise ValueError("packed sequences (cu_seqlens) need B == 1")
        N = cu_seqlens.numel() - 1
        if N == 0 and lead[1] > 0:
            raise ValueError("cu_seqlens names no sequence")
    _lin_out("S0", S0, (N, H, q.shape[-1], v.shape[-1]), torch.float32)
    return N, H, decay, heads


def _addresses(index, names, *tensors):
    """Device addresses of contiguous tensors on CUDA device ``index`` (None: no address);
    ``names`` names them for a refusal."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.get_device() != index or not t.is_contiguous():
            name = names.split()[len(out)]
            raise ValueError(f"{name} is on {t.device}, q on cuda:{index}" if t.get_device() != index
                             else f"{name} must be contiguous")
        else:
            out.append(t.data_ptr())
    return out


def _call(index, name, *args):
    """Calls an entry point on CUDA device ``index`` and its current stream (the last argument)."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if rc != 0:
        raise CkdaError(name, rc)


def _on_cuda(q):
    index = q.get_device()
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    return index


def _room(q, workspace, n):
    """A workspace of n bytes when none is given; returns it (to be kept until the call has been
    issued), its address and its bytes."""
    if workspace is None:
        workspace = q.new_empty(n, dtype=torch.uint8)
    return workspace, _addresses(q.get_device(), "workspace", workspace)[0], workspace.numel() * workspace.element_size()


def linattn_fwd_workspace_size(B, T, H, dk, dv, dtype, n_seqs=0) -> int:
    return (_lib or load()).ckda_linattn_fwd_workspace_size(B, T, H, dk, dv, _DT[dtype], n_seqs)


def linattn_fwd(q, k, v, g, S0=None, cu_seqlens=None, o=None, S_T=None, workspace=None,
                want_o: bool = True, want_state: bool = True):
    """Linear attention with a decay for each head, S_t = exp(g_t) S_{t-1} + k_t v_t^T,
    o_t = S_t^T q_t.  Returns (o, S_T) (either None when not wanted).

    q [B,T,Hq,dk], k [B,T,Hk,dk], v [B,T,Hv,dv] in one dtype (float32 or bfloat16); g: log
    decays <= 0, float32 [B,T,H], or [H] for fixed ones; Hq, Hk and Hv divide H; S0 [N,H,dk,dv]
    float32 or None; cu_seqlens int32 [N+1] on the device (B == 1) or None.  o [B,T,H,dv]."""
    N, H, decay, heads = check_linattn_args(q, k, v, g, S0, cu_seqlens)
    B, T, _, dk = q.shape
    dv, n_seqs = v.shape[-1], 0 if cu_seqlens is None else N
    _lin_out("o", o, (B, T, H, dv), q.dtype)
    _lin_out("S_T", S_T, (N, H, dk, dv), torch.float32)
    index = _on_cuda(q)
    if not want_o:
        o = None
    elif o is None:
        o = q.new_empty((B, T, H, dv))
    if not want_state:
        S_T = None
    elif S_T is None:
        S_T = q.new_empty((N, H, dk, dv), dtype=torch.float32)
    workspace, wp, wn = _room(q, workspace, linattn_fwd_workspace_size(B, T, H, dk, dv, q.dtype, n_seqs))
    p = _addresses(index, "q k v g S0 cu_seqlens o S_T", q, k, v, g, S0, cu_seqlens, o, S_T)
    _call(index, "ckda_linattn_fwd", *p[:6], n_seqs, B, T, H, *heads, dk, dv, decay, _DT[q.dtype], *p[6:], wp, wn)
    return o, S_T


def linattn_bwd_workspace_size(B, T, H, Hq, Hk, Hv, dk, dv, decay, dtype, n_seqs=0) -> int:
    return (_lib or load()).ckda_linattn_bwd_workspace_size(B, T, H, Hq, Hk, Hv, dk, dv, decay,
                                                            _DT[dtype], n_seqs)


def linattn_bwd(q, k, v, g, S0=None, cu_seqlens=None, dO=None, dS_T=None, want_dS0: bool = True,
                workspace=None, grads=None):
    """Backward of ``linattn_fwd``: gradients of sum(dO * o) + sum(dS_T * S_T).

    Returns (dq, dk, dv, dg, dS0): dq, dk, dv as q, k, v; dg as g; dS0 [N,H,dk,dv] float32
    (None when not wanted).  dO [B,T,H,dv] in q's dtype or None (zero); dS_T [N,H,dk,dv]
    float32 or None (zero).  ``grads`` may supply the five output tensors."""
    N, H, decay, heads = check_linattn_args(q, k, v, g, S0, cu_seqlens)
    B, T, _, dk = q.shape
    dv, n_seqs, state = v.shape[-1], 0 if cu_seqlens is None else N, (N, H, dk, v.shape[-1])
    _lin_out("dO", dO, (B, T, H, dv), q.dtype)
    _lin_out("dS_T", dS_T, state, torch.float32)
    if grads is not None:
        for name, t, like in zip(("dq", "dk", "dv", "dg"), grads, (q, k, v, g)):
            if t is None:
                raise ValueError(f"{name} buffer missing")
            _lin_out(name, t, like.shape, like.dtype)
        if want_dS0 and grads[4] is None:
            raise ValueError("dS0 buffer missing")
        _lin_out("dS0", grads[4], state, torch.float32)
    index = _on_cuda(q)
    if grads is None:
        gq, gk, gv, gg = (t.new_empty(t.shape) for t in (q, k, v, g))
        gS0 = q.new_empty(state, dtype=torch.float32) if want_dS0 else None
    else:
        gq, gk, gv, gg, gS0 = grads
        gS0 = gS0 if want_dS0 else None
    workspace, wp, wn = _room(q, workspace, linattn_bwd_workspace_size(
        B, T, H, *heads, dk, dv, decay, q.dtype, n_seqs))
    p = _addresses(index, "q k v g S0 cu_seqlens dO dS_T dq dk dv dg dS0", q, k, v, g, S0, cu_seqlens, dO, dS_T,
                   gq, gk, gv, gg, gS0)
    _call(index, "ckda_linattn_bwd", *p[:6], n_seqs, B, T, H, *heads, dk, dv, decay, _DT[q.dtype], *p[6:], wp, wn)
    return gq, gk, gv, gg, gS0


def linattn_decode_step(q, k, v, g, S, o=None, want_o: bool = True):
    """One token of ``linattn_fwd``: S [B,H,dk,dv] float32 is updated in place; returns o
    [B,H,dv] (None when not wanted).  q [B,Hq,dk], k [B,Hk,dk], v [B,Hv,dv]; g [B,H] or [H]."""
    qs, dt = q.shape, q.dtype
    if len(qs) != 3:
        raise ValueError(f"q must be [B,Hq,dk], got {tuple(qs)}")
    B, _, dk = qs
    H, decay, heads = _lin_heads(g, qs[:1], (("q", q), ("k", k), ("v", v)))
    _lin_types(q, k, v)
    dv = v.shape[2]
    if S.shape != (B, H, dk, dv) or S.dtype != torch.float32:
        raise ValueError(f"S must be [B,H,dk,dv] = {(B, H, dk, dv)} float32")
    index = _on_cuda(q)
    if not want_o:
        o = None
    elif o is None:
        o = q.new_empty((B, H, dv))
    else:
        _lin_out("o", o, (B, H, dv), dt)
    p = _addresses(index, "q k v g S o", q, k, v, g, S, o)
    _call(index, "ckda_linattn_decode_step", *p[:5], B, H, *heads, dk, dv, decay, _DT[dt], p[5])
    return o


# ------------------------------------------------------------------ rotary positions
def rotary_freqs(dim: int, base: float = 10000.0, scaling: Optional[str] = None,
                 factor: float = 1.0, original_len: int = 4096, fast: float = 32.0,
                 slow: float = 1.0, device=None):
    """(freqs, scale) for ``rotary``: float64 radians per position of dim / 2 channel pairs,
    base^(-2 i / dim), and the factor on the turned channels.

    scaling, for contexts ``factor`` times longer than ``original_len``: "linear" divides every
    frequency by the factor; "base" raises the base by factor^(dim / (dim - 2)), which keeps the
    fastest pair and divides the slowest by the factor; "ramp" divides the pairs that turn fewer
    than ``slow`` times over the original length, keeps those that turn more than ``fast`` times,
    blends between, and scales by 0.1 ln(factor) + 1."""
    _need(dim >= 0 and dim % 2 == 0, f"dim must be even, got {dim}")
    _need(scaling in (None, "linear", "base", "ramp"), f"unknown scaling {scaling!r}")
    _need(factor >= 1.0, f"factor must be at least 1, got {factor}")
    _need(scaling != "base" or dim > 2, "scaling 'base' needs more than one pair")
    i = torch.arange(dim // 2, dtype=torch.float64)
    if scaling == "base":
        base = base * factor ** (dim / (dim - 2))
    f = torch.pow(torch.tensor(float(base), dtype=torch.float64), -2.0 * i / max(dim, 1))
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "ramp":
        turns = original_len * f / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f / factor * (1.0 - keep) + f * keep
        scale = 0.1 * math.log(factor) + 1.0
    return f.to("cuda" if device is None else device), scale


def rotary(q, k, pos, freqs, layout: str = "half", inverse: bool = False, scale: float = 1.0,
           q_out=None, k_out=None):
    """Turns channel pairs of q and k by pos * freqs (one launch); returns (q_out, k_out).

    q [*lead,Hq,d], k [*lead,Hk,d] or None, float32 or bfloat16; pos int32 or int64 [*lead];
    freqs float64 [n], 2 n <= d: pair i is channels (i, i + n) ("half") or (2 i, 2 i + 1)
    ("interleaved"); channels from 2 n on are copied.  ``inverse`` turns back (with the same
    scale: the gradient).  An output may be its input."""
    if layout not in ROTARY_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROTARY_LAYOUTS)}, got {layout!r}")
    if q.dim() < 2:
        raise ValueError(f"q must be [*lead,Hq,d], got {tuple(q.shape)}")
    if q.dtype not in _DT:
        raise ValueError(f"q must be float32 or bfloat16, got {q.dtype}")
    lead, d = q.shape[:-2], q.shape[-1]
    if k is not None and (k.dim() != q.dim() or k.shape[:-2] != lead or k.shape[-1] != d or k.dtype != q.dtype):
        raise ValueError(f"k must be {tuple(lead) + ('Hk', d)} in q's dtype, got {tuple(k.shape)}, {k.dtype}")
    if pos.shape != lead or pos.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"pos must be {tuple(lead)} int32 or int64, got {tuple(pos.shape)}, {pos.dtype}")
    if freqs.dim() != 1 or freqs.dtype != torch.float64 or 2 * freqs.shape[0] > d:
        raise ValueError(f"freqs must be float64 [n] with 2 n <= {d}, got {tuple(freqs.shape)}, {freqs.dtype}")
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    if q_out is not None:
        _lin_out("q_out", q_out, q.shape, q.dtype)
    if k is not None and k_out is not None:
        _lin_out("k_out", k_out, k.shape, k.dtype)
    index = _on_cuda(q)
    if q_out is None:
        q_out = q.new_empty(q.shape)
    if k is not None and k_out is None:
        k_out = k.new_empty(k.shape)
    p = _addresses(index, "q k pos freqs q_out k_out", q, k, pos, freqs, q_out, k_out)
    _call(index, "ckda_rotary", *p[:4], pos.numel(), q.shape[-2], 0 if k is None else k.shape[-2], d, freqs.shape[0],
          ROTARY_LAYOUTS[layout], pos.dtype == torch.int64, scale, inverse, _DT[q.dtype], p[4], p[5])
    return q_out, k_out
