"""The operators around the gated delta rule: the short causal convolution, the
selective state space scan, the single-token forms and the norms around a
block (``include/gdr.h``).  Argument marshalling only, as in the package's main
module, which re-exports every name; all arguments are checked for device,
type, shape and layout before the library is called, and a check that fails
raises ``ValueError`` with nothing enqueued.

Outputs and workspaces are allocated on the stream the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes

import numpy as np
import torch

from . import _check, load

__all__ = ("sconv_workspace_bytes", "sconv_fwd", "sconv_bwd", "sconv_step", "ssm_workspace_bytes", "ssm_fwd", "ssm_step",
           "kda_step", "gdn_step", "norm_workspace_bytes", "norm_fwd", "norm_bwd")

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACT = {"silu": 0, "sigmoid": 1}
_F32 = torch.float32
_BF16 = torch.bfloat16
_I32 = torch.int32


def _fail(where, what):
    raise ValueError(f"{where}: {what}")


def _on(where, dev, **tensors):
    """Every given tensor lives on `dev`."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            _fail(where, f"{name} is on {t.device}, expected {dev}")


def _device(where, t):
    dev = t.device
    if dev.type != "cuda":
        _fail(where, f"tensors must be on a CUDA device, got {dev}")
    if dev.index != torch.cuda.current_device():
        _fail(where, f"tensors are on {dev}, the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _dense(where, name, t, dtype, shape):
    """A dense tensor of exactly this type and shape; its address (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape:
        _fail(where, f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if not t.is_contiguous():
        _fail(where, f"{name} must be contiguous")
    return t.data_ptr()


def _on_stream(stream):
    """The context that allocates on `stream` (None: the current one)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raw(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream


def _pack(where, cu_seqlens, cu_seqlens_host, dev):
    """(device pointer, host pointer, documents, the host array kept alive)."""
    host = cu_seqlens_host
    if hasattr(host, "detach"):
        host = host.detach().cpu().numpy()
    host = np.ascontiguousarray(host, dtype=np.int32)
    if host.ndim != 1 or host.shape[0] < 1:
        _fail(where, "cu_seqlens_host must be one-dimensional with at least one entry")
    n = host.shape[0] - 1
    if cu_seqlens.dtype is not _I32 or cu_seqlens.shape != (n + 1,) or not cu_seqlens.is_contiguous():
        _fail(where, f"cu_seqlens must be a contiguous int32 tensor of {n + 1} entries")
    return cu_seqlens.data_ptr(), host.ctypes.data, n, host


def _slots(where, slots, batch, dev):
    if slots is None:
        return 0
    if slots.dtype is not _I32 or slots.shape != (batch,) or not slots.is_contiguous():
        _fail(where, f"slots must be a contiguous int32 tensor of {batch} entries")
    return slots.data_ptr()


def _scratch(scratch, need, dev):
    if scratch is None:
        scratch = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    return scratch


# ---------------------------------------------------------------------------
# Short causal convolution
# ---------------------------------------------------------------------------
def _conv_args(where, x, weight, bias):
    if x.dim() != 2:
        _fail(where, f"x has shape {tuple(x.shape)}, expected [tokens, channels]")
    dt = _DTYPE.get(x.dtype)
    if dt is None:
        _fail(where, f"x is {x.dtype}; bfloat16, float16 and float32 are supported")
    C = x.shape[1]
    if weight.dim() != 2 or weight.shape[0] != C or not 2 <= weight.shape[1] <= 4:
        _fail(where, f"weight has shape {tuple(weight.shape)}, expected [{C}, 2 to 4]")
    if weight.dtype is not x.dtype and weight.dtype is not _F32:
        _fail(where, f"weight is {weight.dtype}, expected {x.dtype} or float32")
    W = weight.shape[1]
    wp = _dense(where, "weight", weight, weight.dtype, (C, W))
    bp = _dense(where, "bias", bias, weight.dtype, (C,))
    return dt, C, W, wp, bp, _DTYPE[weight.dtype]


def _rows(where, name, t):
    """Row stride of a 2-D tensor with dense rows."""
    if t.stride(1) != 1 and t.shape[1] > 1:
        _fail(where, f"{name} must have dense rows")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def sconv_workspace_bytes(T: int, C: int, W: int) -> int:
    """Scratch bytes of sconv_bwd; host only."""
    n = ctypes.c_size_t(0)
    _check(load().sconv_workspace_bytes(T, C, W, ctypes.byref(n)), "sconv_workspace_bytes")
    return n.value


def sconv_fwd(x, weight, bias, cu_seqlens, cu_seqlens_host, s0=None, silu=True, out=None, st=None, want_st=True,
              stream=None):
    """Short causal depthwise convolution over packed documents.

    x [T, C] (bf16, fp16 or fp32; rows may be strided), weight [C, W] with W of
    2 to 4 and bias [C] or None (x's type or fp32), s0 [N, W-1, C] the
    documents' start states or None.  Returns (out [T, C], st [N, W-1, C]): st
    holds each document's last W - 1 inputs (None when not wanted)."""
    dev = _device("sconv_fwd", x)
    dt, C, W, wp, bp, wdt = _conv_args("sconv_fwd", x, weight, bias)
    T = x.shape[0]
    cu, cuh, n, keep = _pack("sconv_fwd", cu_seqlens, cu_seqlens_host, dev)
    _on("sconv_fwd", dev, weight=weight, bias=bias, cu_seqlens=cu_seqlens, s0=s0, out=out, st=st)
    with _on_stream(stream):
        if out is None:
            out = torch.empty((T, C), dtype=x.dtype, device=dev)
        if st is None and want_st:
            st = torch.empty((n, W - 1, C), dtype=x.dtype, device=dev)
    state = (n, W - 1, C)
    _check(load().sconv_fwd(dt, x.data_ptr(), _rows("sconv_fwd", "x", x), wp, bp, wdt, cu, cuh, n, T, C, W,
                            1 if silu else 0, _dense("sconv_fwd", "s0", s0, x.dtype, state),
                            _dense("sconv_fwd", "out", out, x.dtype, (T, C)),
                            _dense("sconv_fwd", "st", st, x.dtype, state), _raw(stream, dev)), "sconv_fwd")
    return out, st


def sconv_bwd(x, weight, bias, cu_seqlens, cu_seqlens_host, dout, s0=None, dst=None, want_ds0=False, silu=True,
              scratch=None, grads=None, stream=None):
    """Gradients of sconv_fwd from dout [T, C] (and dst, the gradient of st).
    Returns a dict with dx, dweight (fp32), dbias (fp32, None without a bias)
    and, when wanted, ds0; `grads` may bring preallocated tensors."""
    dev = _device("sconv_bwd", x)
    dt, C, W, wp, bp, wdt = _conv_args("sconv_bwd", x, weight, bias)
    T = x.shape[0]
    cu, cuh, n, keep = _pack("sconv_bwd", cu_seqlens, cu_seqlens_host, dev)
    if dout.dtype is not x.dtype or dout.shape != x.shape:
        _fail("sconv_bwd", f"dout is {dout.dtype} {tuple(dout.shape)}, expected {x.dtype} {tuple(x.shape)}")
    got = dict(grads or {})
    need = sconv_workspace_bytes(T, C, W)
    with _on_stream(stream):
        if "dx" not in got:
            got["dx"] = torch.empty((T, C), dtype=x.dtype, device=dev)
        if "dweight" not in got:
            got["dweight"] = torch.empty((C, W), dtype=_F32, device=dev)
        if bias is None:
            got["dbias"] = None
        elif "dbias" not in got:
            got["dbias"] = torch.empty((C,), dtype=_F32, device=dev)
        if want_ds0 and "ds0" not in got:
            got["ds0"] = torch.empty((n, W - 1, C), dtype=x.dtype, device=dev)
        scratch = _scratch(scratch, need, dev)
    ds0 = got.get("ds0")
    _on("sconv_bwd", dev, weight=weight, bias=bias, cu_seqlens=cu_seqlens, s0=s0, dout=dout, dst=dst, scratch=scratch,
        dx=got["dx"], dweight=got["dweight"], dbias=got["dbias"], ds0=ds0)
    state = (n, W - 1, C)
    _check(load().sconv_bwd(dt, x.data_ptr(), _rows("sconv_bwd", "x", x), wp, bp, wdt, cu, cuh, n, T, C, W,
                            1 if silu else 0, _dense("sconv_bwd", "s0", s0, x.dtype, state), dout.data_ptr(),
                            _rows("sconv_bwd", "dout", dout), _dense("sconv_bwd", "dst", dst, x.dtype, state),
                            _dense("sconv_bwd", "dx", got["dx"], x.dtype, (T, C)),
                            _dense("sconv_bwd", "dweight", got["dweight"], _F32, (C, W)),
                            _dense("sconv_bwd", "dbias", got["dbias"], _F32, (C,)),
                            _dense("sconv_bwd", "ds0", ds0, x.dtype, state), scratch.data_ptr(),
                            scratch.numel() * scratch.element_size(), _raw(stream, dev)), "sconv_bwd")
    return got


def sconv_step(x, weight, bias, state, slots=None, silu=True, out=None, stream=None):
    """One token of each sequence: x [B, C], state [S, W-1, C] updated in place,
    slots int32 [B] (None: row b uses state b; a slot outside [0, S) makes the
    row inactive).  Returns out [B, C]."""
    dev = _device("sconv_step", x)
    dt, C, W, wp, bp, wdt = _conv_args("sconv_step", x, weight, bias)
    B = x.shape[0]
    _on("sconv_step", dev, weight=weight, bias=bias, state=state, slots=slots, out=out)
    if out is None:
        with _on_stream(stream):
            out = torch.empty((B, C), dtype=x.dtype, device=dev)
    S = state.shape[0]
    _check(load().sconv_step(dt, x.data_ptr(), _rows("sconv_step", "x", x), wp, bp, wdt,
                             _dense("sconv_step", "state", state, x.dtype, (S, W - 1, C)),
                             _slots("sconv_step", slots, B, dev), B, S, C, W, 1 if silu else 0,
                             _dense("sconv_step", "out", out, x.dtype, (B, C)), _raw(stream, dev)), "sconv_step")
    return out


# ---------------------------------------------------------------------------
# Selective state space scan
# ---------------------------------------------------------------------------
def _heads(where, name, t, T):
    """Token stride of a [T, heads, dim] tensor whose (heads, dim) are dense."""
    if t.dim() != 3 or t.shape[0] != T:
        _fail(where, f"{name} has shape {tuple(t.shape)}, expected [{T}, heads, dim]")
    if t.dtype is not _BF16:
        _fail(where, f"{name} is {t.dtype}, expected bfloat16")
    _, h, d = t.shape
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        _fail(where, f"{name} must be dense within a token")
    return s[0] if T > 1 else h * d


def _ssm_args(where, x, dt, A, B, C, D, dt_bias):
    if x.dim() != 3:
        _fail(where, f"x has shape {tuple(x.shape)}, expected [tokens, heads, head dim]")
    T, H, P = x.shape
    ldx, ldb, ldc = _heads(where, "x", x, T), _heads(where, "B", B, T), _heads(where, "C", C, T)
    if B.shape != C.shape:
        _fail(where, f"B has shape {tuple(B.shape)} and C {tuple(C.shape)}")
    G, NS = B.shape[1:]
    if dt.shape != (T, H) or dt.dtype not in (_BF16, _F32) or (H > 1 and dt.stride(1) != 1):
        _fail(where, f"dt is {dt.dtype} {tuple(dt.shape)}, expected bfloat16 or float32 [{T}, {H}] with dense rows")
    head = (H,)
    if G < 1 or H % G:
        _fail(where, f"{H} heads do not share {G} groups of B and C evenly")
    return (T, H, P, G, NS, ldx, ldb, ldc, dt.stride(0) if T > 1 else H, _dense(where, "A", A, _F32, head),
            _dense(where, "D", D, _F32, head), _dense(where, "dt_bias", dt_bias, _F32, head))


def ssm_workspace_bytes(T: int, H: int, P: int, G: int, NS: int, cu_seqlens_host) -> int:
    """Scratch bytes of ssm_fwd; host only."""
    host = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    n = ctypes.c_size_t(0)
    _check(load().ssm_workspace_bytes(T, H, P, G, NS, host.shape[0] - 1, host.ctypes.data, ctypes.byref(n)),
           "ssm_workspace_bytes")
    return n.value


def ssm_fwd(x, dt, A, B, C, cu_seqlens, cu_seqlens_host, D=None, dt_bias=None, softplus=True, h0=None, out=None,
            ht=None, want_ht=True, scratch=None, stream=None):
    """Selective state space scan over packed documents.

    x bf16 [T, H, P]; dt bf16 or fp32 [T, H]; A (negative), D, dt_bias fp32
    [H]; B, C bf16 [T, G, NS], shared by the H / G heads of a group; h0 fp32 [N,
    H, NS, P] or None.  x, B, C and dt may be slices of wider rows.  Returns
    (out bf16 [T, H, P], ht fp32 [N, H, NS, P] or None)."""
    where = "ssm_fwd"
    dev = _device(where, x)
    T, H, P, G, NS, ldx, ldb, ldc, lddt, Ap, Dp, bp = _ssm_args(where, x, dt, A, B, C, D, dt_bias)
    cu, cuh, n, keep = _pack(where, cu_seqlens, cu_seqlens_host, dev)
    lib = load()
    need = ctypes.c_size_t(0)
    _check(lib.ssm_workspace_bytes(T, H, P, G, NS, n, cuh, ctypes.byref(need)), where)
    with _on_stream(stream):
        if out is None:
            out = torch.empty((T, H, P), dtype=_BF16, device=dev)
        if ht is None and want_ht:
            ht = torch.empty((n, H, NS, P), dtype=_F32, device=dev)
        if scratch is None and need.value:
            scratch = _scratch(None, need.value, dev)
    _on(where, dev, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, cu_seqlens=cu_seqlens, h0=h0, out=out, ht=ht,
        scratch=scratch)
    state = (n, H, NS, P)
    _check(lib.ssm_fwd(x.data_ptr(), ldx, dt.data_ptr(), _DTYPE[dt.dtype], lddt, Ap, B.data_ptr(), ldb, C.data_ptr(),
                       ldc, Dp, bp, 1 if softplus else 0, cu, cuh, n, T, H, P, G, NS,
                       _dense(where, "h0", h0, _F32, state), _dense(where, "out", out, _BF16, (T, H, P)),
                       _dense(where, "ht", ht, _F32, state), 0 if scratch is None else scratch.data_ptr(),
                       0 if scratch is None else scratch.numel() * scratch.element_size(), _raw(stream, dev)), where)
    return out, ht


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, softplus=True, slots=None, out=None, stream=None):
    """One token of each sequence through the scan: x [B, H, P], dt [B, H], B and
    C [B, G, NS], state fp32 [S, H, NS, P] updated in place; slots as in
    sconv_step.  Returns out bf16 [B, H, P]."""
    where = "ssm_step"
    dev = _device(where, x)
    T, H, P, G, NS, ldx, ldb, ldc, lddt, Ap, Dp, bp = _ssm_args(where, x, dt, A, B, C, D, dt_bias)
    _on(where, dev, dt=dt, A=A, B=B, C=C, D=D, dt_bias=dt_bias, state=state, slots=slots, out=out)
    if out is None:
        with _on_stream(stream):
            out = torch.empty((T, H, P), dtype=_BF16, device=dev)
    S = state.shape[0]
    _check(load().ssm_step(x.data_ptr(), ldx, dt.data_ptr(), _DTYPE[dt.dtype], lddt, Ap, B.data_ptr(), ldb,
                           C.data_ptr(), ldc, Dp, bp, 1 if softplus else 0,
                           _dense(where, "state", state, _F32, (S, H, NS, P)), _slots(where, slots, T, dev), T, S, H,
                           P, G, NS, _dense(where, "out", out, _BF16, (T, H, P)), _raw(stream, dev)), where)
    return out


# ---------------------------------------------------------------------------
# One token of the gated delta rule
# ---------------------------------------------------------------------------
def _delta_step(variant, q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream):
    where = variant + "_step"
    dev = _device(where, q)
    if q.dim() != 3 or v.dim() != 3 or q.shape[2] != 128:
        _fail(where, f"q has shape {tuple(q.shape)} and v {tuple(v.shape)}, expected [batch, heads, 128]")
    B, Hqk, _ = q.shape
    HV, S = v.shape[1], state.shape[0]
    kda = variant == "kda"
    if kda and Hqk != HV:
        _fail(where, f"q and k have {Hqk} heads and v has {HV}; KDA needs the same count")
    if HV % max(Hqk, 1):
        _fail(where, f"{HV} value heads do not share {Hqk} q/k heads evenly")
    _on(where, dev, k=k, v=v, g=g, beta=beta, state=state, slots=slots, out=out)
    if out is None:
        with _on_stream(stream):
            out = torch.empty((B, HV, 128), dtype=_BF16, device=dev)
    heads, vals = (B, Hqk, 128), (B, HV, 128)
    ptrs = (_dense(where, "q", q, _BF16, heads), _dense(where, "k", k, _BF16, heads), _dense(where, "v", v, _BF16, vals),
            _dense(where, "g", g, _F32, vals if kda else (B, HV)),
            _dense(where, "beta", beta, _BF16 if kda else _F32, (B, HV)),
            _dense(where, "state", state, _F32, (S, HV, 128, 128)), _slots(where, slots, B, dev), B, S)
    tail = (scale, 1 if qk_l2norm else 0, _dense(where, "out", out, _BF16, vals), _raw(stream, dev))
    if kda:
        _check(load().kda_step(*ptrs, HV, *tail), where)
    else:
        _check(load().gdn_step(*ptrs, Hqk, HV, *tail), where)
    return out


def kda_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through KDA: q, k, v bf16 [B, H, 128], g fp32
    [B, H, 128], beta bf16 [B, H], state fp32 [S, H, 128, 128] (a forward's ht)
    updated in place; slots as in sconv_step.  Returns out bf16 [B, H, 128]."""
    return _delta_step("kda", q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream)


def gdn_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through grouped GDN: q, k bf16 [B, Hqk, 128], v
    bf16 [B, HV, 128], g, beta fp32 [B, HV], state fp32 [S, HV, 128, 128]."""
    return _delta_step("gdn", q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream)


# ---------------------------------------------------------------------------
# Norms around a block
# ---------------------------------------------------------------------------
def _row_strides(where, name, t, x):
    """(address, outer stride, inner stride) of a row tensor shaped like x: [..., D]
    viewed as [R0, R1, D] with dense rows."""
    if t is None:
        return 0, 0, 0
    if t is not x and (t.shape != x.shape or t.dtype is not x.dtype):
        _fail(where, f"{name} is {t.dtype} {tuple(t.shape)}, expected {x.dtype} {tuple(x.shape)}")
    s = t.stride()
    D = t.shape[-1]
    if s[-1] != 1 and D > 1:
        _fail(where, f"{name} must have dense rows")
    nd = t.dim()
    if nd == 1:
        return t.data_ptr(), D, D
    if nd == 2:
        return t.data_ptr(), s[0], D
    if nd == 3:
        return t.data_ptr(), s[0], s[1]
    if not t.is_contiguous():
        _fail(where, f"{name} has {nd} dimensions and must be contiguous")
    return t.data_ptr(), D * t.shape[-2], D


def _norm_args(where, x, weight, post_weight, gate, act, residual):
    dt = _DTYPE.get(x.dtype)
    if dt is None:
        _fail(where, f"x is {x.dtype}; bfloat16, float16 and float32 are supported")
    if x.dim() < 1 or not 1 <= x.shape[-1] <= 16384:
        _fail(where, f"x has shape {tuple(x.shape)}; rows of 1 to 16384 elements are supported")
    if act not in _ACT:
        _fail(where, f"act {act!r}, expected 'silu' or 'sigmoid'")
    if weight is None and post_weight is None and residual is None:
        _fail(where, "one of weight, post_weight and residual is needed")
    D = x.shape[-1]
    R1 = x.shape[-2] if x.dim() >= 3 else 1
    R0 = x.numel() // (R1 * D) if R1 else 0
    w = weight if weight is not None else post_weight
    wt = x.dtype if w is None else w.dtype
    if wt is not x.dtype and wt is not _F32:
        _fail(where, f"weights are {wt}, expected {x.dtype} or float32")
    return (dt, R0, max(R1, 1), D, _row_strides(where, "x", x, x), _row_strides(where, "gate", gate, x),
            _row_strides(where, "residual", residual, x), _dense(where, "post_weight", post_weight, wt, (D,)),
            _dense(where, "weight", weight, wt, (D,)), _DTYPE[wt])


def norm_workspace_bytes(D: int) -> int:
    """Scratch bytes of norm_bwd for rows of D elements; host only."""
    n = ctypes.c_size_t(0)
    _check(load().norm_workspace_bytes(D, ctypes.byref(n)), "norm_workspace_bytes")
    return n.value


def norm_fwd(x, weight=None, post_weight=None, gate=None, act="silu", residual=None, res_scale=1.0, eps=1e-6, h=None,
             y=None, stream=None):
    """The norms around a block, its gate and its scaled residual, in one pass:

        u = x, or RMSNorm(x) post_weight;  u = u act(gate);
        h = residual + res_scale u, or u;  y = RMSNorm(h) weight

    on rows x [..., D] (bf16, fp16 or fp32; two leading dimensions may be
    strided); gate and residual are shaped like x, the weights [D] (x's type or
    fp32).  Returns (h, y): h is None when neither a residual nor a missing
    `weight` makes it an output, y is None without `weight`."""
    where = "norm_fwd"
    dev = _device(where, x)
    dt, R0, R1, D, xs, gs, rs, pp, wp, wdt = _norm_args(where, x, weight, post_weight, gate, act, residual)
    _on(where, dev, weight=weight, post_weight=post_weight, gate=gate, residual=residual, h=h, y=y)
    with _on_stream(stream):
        if h is None and (residual is not None or weight is None):
            h = torch.empty(x.shape, dtype=x.dtype, device=dev)
        if y is None and weight is not None:
            y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    _check(load().norm_fwd(dt, R0, R1, D, *xs, *gs, _ACT[act], *rs, res_scale, pp, wp, wdt, eps,
                           _dense(where, "h", h, x.dtype, x.shape), _dense(where, "y", y, x.dtype, x.shape),
                           _raw(stream, dev)), where)
    return h, y


def norm_bwd(x, weight=None, post_weight=None, gate=None, act="silu", residual=None, res_scale=1.0, eps=1e-6, dh=None,
             dy=None, scratch=None, grads=None, stream=None):
    """Gradients of norm_fwd from dh and dy (the gradients of h and y; either may
    be None).  Returns a dict with dx and, for the arguments given, dgate,
    dresidual, dweight and dpost_weight (fp32); `grads` may bring preallocated
    tensors.  Where u = x and res_scale = 1, dx and dresidual are one tensor."""
    where = "norm_bwd"
    dev = _device(where, x)
    dt, R0, R1, D, xs, gs, rs, pp, wp, wdt = _norm_args(where, x, weight, post_weight, gate, act, residual)
    if dh is None and dy is None:
        _fail(where, "one of dh and dy is needed")
    if dy is not None and weight is None:
        _fail(where, "dy without weight")
    got = dict(grads or {})
    same = residual is not None and post_weight is None and gate is None and res_scale == 1.0 and not grads
    need = norm_workspace_bytes(D)
    with _on_stream(stream):
        for name, given, like in (("dx", x, x), ("dgate", gate, x), ("dresidual", residual, x)):
            if given is not None and name not in got:
                got[name] = got["dx"] if same and name == "dresidual" else torch.empty(x.shape, dtype=x.dtype, device=dev)
        for name, given in (("dweight", weight), ("dpost_weight", post_weight)):
            if given is not None and name not in got:
                got[name] = torch.empty((D,), dtype=_F32, device=dev)
        scratch = _scratch(scratch, need, dev)
    _on(where, dev, weight=weight, post_weight=post_weight, gate=gate, residual=residual, dh=dh, dy=dy, scratch=scratch,
        **got)
    rows = tuple(0 if same and n == "dresidual" else _dense(where, n, got.get(n), x.dtype, x.shape)
                 for n in ("dx", "dgate", "dresidual"))
    _check(load().norm_bwd(dt, R0, R1, D, *xs, *gs, _ACT[act], *rs, res_scale, pp, wp, wdt, eps,
                           *_row_strides(where, "dh", dh, x), *_row_strides(where, "dy", dy, x), *rows,
                           _dense(where, "dweight", got.get("dweight"), _F32, (D,)),
                           _dense(where, "dpost_weight", got.get("dpost_weight"), _F32, (D,)), scratch.data_ptr(),
                           scratch.numel() * scratch.element_size(), _raw(stream, dev)), where)
    return got
