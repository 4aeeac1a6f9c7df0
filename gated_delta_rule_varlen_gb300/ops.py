"""The operators around the gated delta rule: the short causal convolution, the
selective state space scan, the single-token forms and the norms around a
block (``include/gdr.h``).  Argument marshalling only, as in the package's main
module, which re-exports every name; all arguments are checked for device,
type, shape and layout before the library is called, and a check that fails
raises ``ValueError`` with nothing enqueued.

Outputs and workspaces are allocated on the stream the call runs on.
"""
from __future__ import annotations

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
_U8 = torch.uint8
_NONE3 = (0, 0, 0)

_new = torch.empty
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _fail(where, what):
    raise ValueError(f"{where}: {what}")


def _device(where, t):
    """Index of the current CUDA device, which must hold `t`."""
    if not t.is_cuda:
        _fail(where, f"tensors must be on a CUDA device, got {t.device}")
    index = t.get_device()
    if index != _current_device():
        _fail(where, f"tensors are on {t.device}, the current device is cuda:{_current_device()}")
    return index


def _on(where, dev, name, t):
    if t.get_device() != dev:
        _fail(where, f"{name} is on {t.device}, expected cuda:{dev}")


def _dense(where, dev, name, t, dtype, shape):
    """The address of a dense tensor of exactly this type and shape (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape:
        _fail(where, f"{name} is {t.dtype} {tuple(t.shape)}, expected {dtype} {tuple(shape)}")
    if not t.is_contiguous():
        _fail(where, f"{name} must be contiguous")
    if t.get_device() != dev:
        _fail(where, f"{name} is on {t.device}, expected cuda:{dev}")
    return t.data_ptr()


def _empty(like, stream, shape, dtype):
    """Allocated on the stream the call runs on."""
    if stream is None:
        return _new(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return _new(shape, dtype=dtype, device=like.device)


def _raw(stream, dev):
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _pack(where, dev, cu_seqlens, cu_seqlens_host):
    """(device pointer, host pointer, documents, the host array, kept alive)."""
    host = cu_seqlens_host
    if type(host) is not np.ndarray or host.dtype != np.int32 or not host.flags.c_contiguous:
        if hasattr(host, "detach"):
            host = host.detach().cpu().numpy()
        host = np.ascontiguousarray(host, dtype=np.int32)
    if host.ndim != 1 or host.shape[0] < 1:
        _fail(where, "cu_seqlens_host must be one-dimensional with at least one entry")
    n = host.shape[0] - 1
    return _dense(where, dev, "cu_seqlens", cu_seqlens, _I32, (n + 1,)), host.ctypes.data, n, host


def _scratch(where, dev, scratch, need, like, stream):
    """(the tensor, kept alive; its address; its bytes)"""
    if scratch is None:
        scratch = _empty(like, stream, (need if need > 256 else 256,), _U8)
    elif not scratch.is_contiguous() or scratch.get_device() != dev:
        _fail(where, f"scratch must be contiguous and on cuda:{dev}")
    return scratch, scratch.data_ptr(), scratch.numel() * scratch.element_size()


# ---------------------------------------------------------------------------
# Short causal convolution
# ---------------------------------------------------------------------------
def _conv_args(where, dev, x, weight, bias):
    shape, wt = weight.shape, weight.dtype
    if x.dim() != 2:
        _fail(where, f"x has shape {tuple(x.shape)}, expected [tokens, channels]")
    dt = _DTYPE.get(x.dtype)
    if dt is None:
        _fail(where, f"x is {x.dtype}; bfloat16, float16 and float32 are supported")
    T, C = x.shape
    if len(shape) != 2 or shape[0] != C or not 2 <= shape[1] <= 4:
        _fail(where, f"weight has shape {tuple(shape)}, expected [{C}, 2 to 4]")
    if wt is not x.dtype and wt is not _F32:
        _fail(where, f"weight is {wt}, expected {x.dtype} or float32")
    return (dt, T, C, shape[1], _dense(where, dev, "weight", weight, wt, shape),
            0 if bias is None else _dense(where, dev, "bias", bias, wt, (C,)), _DTYPE[wt])


def _rows(where, name, t):
    """Row stride of a 2-D tensor with dense rows."""
    s = t.stride()
    if s[1] != 1 and t.shape[1] > 1:
        _fail(where, f"{name} must have dense rows")
    return s[0] if t.shape[0] > 1 else t.shape[1]


def sconv_workspace_bytes(T: int, C: int, W: int) -> int:
    """Scratch bytes of sconv_bwd; host only."""
    n = ctypes.c_size_t(0)
    _check(_library().sconv_workspace_bytes(T, C, W, ctypes.byref(n)), "sconv_workspace_bytes")
    return n.value


def sconv_fwd(x, weight, bias, cu_seqlens, cu_seqlens_host, s0=None, silu=True, out=None, st=None, want_st=True,
              stream=None):
    """Short causal depthwise convolution over packed documents.

    x [T, C] (bf16, fp16 or fp32; rows may be strided), weight [C, W] with W of
    2 to 4 and bias [C] or None (x's type or fp32), s0 [N, W-1, C] the
    documents' start states or None.  Returns (out [T, C], st [N, W-1, C]): st
    holds each document's last W - 1 inputs (None when not wanted)."""
    where = "sconv_fwd"
    dev = _device(where, x)
    dt, T, C, W, wp, bp, wdt = _conv_args(where, dev, x, weight, bias)
    cu, cuh, n, keep = _pack(where, dev, cu_seqlens, cu_seqlens_host)
    t, state = x.dtype, (n, W - 1, C)
    if out is None:
        out = _empty(x, stream, (T, C), t)
    if st is None and want_st:
        st = _empty(x, stream, state, t)
    code = _library().sconv_fwd(dt, x.data_ptr(), _rows(where, "x", x), wp, bp, wdt, cu, cuh, n, T, C, W,
                                1 if silu else 0, _dense(where, dev, "s0", s0, t, state),
                                _dense(where, dev, "out", out, t, (T, C)), _dense(where, dev, "st", st, t, state),
                                _raw(stream, dev))
    if code:
        _check(code, where)
    return out, st


def sconv_bwd(x, weight, bias, cu_seqlens, cu_seqlens_host, dout, s0=None, dst=None, want_ds0=False, silu=True,
              scratch=None, grads=None, stream=None):
    """Gradients of sconv_fwd from dout [T, C] (and dst, the gradient of st).
    Returns a dict with dx, dweight (fp32), dbias (fp32, None without a bias)
    and, when wanted, ds0; `grads` may bring preallocated tensors."""
    where = "sconv_bwd"
    dev = _device(where, x)
    dt, T, C, W, wp, bp, wdt = _conv_args(where, dev, x, weight, bias)
    cu, cuh, n, keep = _pack(where, dev, cu_seqlens, cu_seqlens_host)
    t, state = x.dtype, (n, W - 1, C)
    if dout.dtype is not t or dout.shape != x.shape:
        _fail(where, f"dout is {dout.dtype} {tuple(dout.shape)}, expected {t} {tuple(x.shape)}")
    _on(where, dev, "dout", dout)
    got = dict(grads or {})
    if "dx" not in got:
        got["dx"] = _empty(x, stream, (T, C), t)
    if "dweight" not in got:
        got["dweight"] = _empty(x, stream, (C, W), _F32)
    if bias is None:
        got["dbias"] = None
    elif "dbias" not in got:
        got["dbias"] = _empty(x, stream, (C,), _F32)
    if want_ds0 and "ds0" not in got:
        got["ds0"] = _empty(x, stream, state, t)
    scratch, sp, sb = _scratch(where, dev, scratch, sconv_workspace_bytes(T, C, W), x, stream)
    code = _library().sconv_bwd(dt, x.data_ptr(), _rows(where, "x", x), wp, bp, wdt, cu, cuh, n, T, C, W,
                                1 if silu else 0, _dense(where, dev, "s0", s0, t, state), dout.data_ptr(),
                                _rows(where, "dout", dout), _dense(where, dev, "dst", dst, t, state),
                                _dense(where, dev, "dx", got["dx"], t, (T, C)),
                                _dense(where, dev, "dweight", got["dweight"], _F32, (C, W)),
                                _dense(where, dev, "dbias", got["dbias"], _F32, (C,)),
                                _dense(where, dev, "ds0", got.get("ds0"), t, state), sp, sb, _raw(stream, dev))
    if code:
        _check(code, where)
    return got


def sconv_step(x, weight, bias, state, slots=None, silu=True, out=None, stream=None):
    """One token of each sequence: x [B, C], state [S, W-1, C] updated in place,
    slots int32 [B] (None: row b uses state b; a slot outside [0, S) makes the
    row inactive).  Returns out [B, C]."""
    where = "sconv_step"
    dev = _device(where, x)
    dt, B, C, W, wp, bp, wdt = _conv_args(where, dev, x, weight, bias)
    t, S = x.dtype, state.shape[0]
    if out is None:
        out = _empty(x, stream, (B, C), t)
        op = out.data_ptr()
    else:
        op = _dense(where, dev, "out", out, t, (B, C))
    code = _library().sconv_step(dt, x.data_ptr(), _rows(where, "x", x), wp, bp, wdt,
                                 _dense(where, dev, "state", state, t, (S, W - 1, C)),
                                 _dense(where, dev, "slots", slots, _I32, (B,)), B, S, C, W, 1 if silu else 0, op,
                                 _raw(stream, dev))
    if code:
        _check(code, where)
    return out


# ---------------------------------------------------------------------------
# Selective state space scan
# ---------------------------------------------------------------------------
def _heads(where, dev, name, t, T):
    """Token stride of a [T, heads, dim] tensor whose (heads, dim) are dense."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != T:
        _fail(where, f"{name} has shape {tuple(shape)}, expected [{T}, heads, dim]")
    if t.dtype is not _BF16:
        _fail(where, f"{name} is {t.dtype}, expected bfloat16")
    _on(where, dev, name, t)
    _, h, d = shape
    s = t.stride()
    if (d > 1 and s[2] != 1) or (h > 1 and s[1] != d):
        _fail(where, f"{name} must be dense within a token")
    return s[0] if T > 1 else h * d


def _ssm_args(where, dev, x, dt, A, B, C, D, dt_bias):
    if x.dim() != 3:
        _fail(where, f"x has shape {tuple(x.shape)}, expected [tokens, heads, head dim]")
    T, H, P = x.shape
    ldx, ldb, ldc = _heads(where, dev, "x", x, T), _heads(where, dev, "B", B, T), _heads(where, dev, "C", C, T)
    if B.shape != C.shape:
        _fail(where, f"B has shape {tuple(B.shape)} and C {tuple(C.shape)}")
    G, NS = B.shape[1:]
    s = dt.stride()
    if dt.shape != (T, H) or dt.dtype not in (_BF16, _F32) or (H > 1 and s[1] != 1):
        _fail(where, f"dt is {dt.dtype} {tuple(dt.shape)}, expected bfloat16 or float32 [{T}, {H}] with dense rows")
    _on(where, dev, "dt", dt)
    head = (H,)
    if G < 1 or H % G:
        _fail(where, f"{H} heads do not share {G} groups of B and C evenly")
    ldt = s[0] if T > 1 else H
    return (T, H, P, G, NS,
            (x.data_ptr(), ldx, dt.data_ptr(), _DTYPE[dt.dtype], ldt, _dense(where, dev, "A", A, _F32, head),
             B.data_ptr(), ldb, C.data_ptr(), ldc, _dense(where, dev, "D", D, _F32, head),
             _dense(where, dev, "dt_bias", dt_bias, _F32, head)))


def ssm_workspace_bytes(T: int, H: int, P: int, G: int, NS: int, cu_seqlens_host) -> int:
    """Scratch bytes of ssm_fwd; host only."""
    host = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    n = ctypes.c_size_t(0)
    _check(_library().ssm_workspace_bytes(T, H, P, G, NS, host.shape[0] - 1, host.ctypes.data, ctypes.byref(n)),
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
    T, H, P, G, NS, args = _ssm_args(where, dev, x, dt, A, B, C, D, dt_bias)
    cu, cuh, n, keep = _pack(where, dev, cu_seqlens, cu_seqlens_host)
    lib, state = _library(), (n, H, NS, P)
    need = ctypes.c_size_t(0)
    _check(lib.ssm_workspace_bytes(T, H, P, G, NS, n, cuh, ctypes.byref(need)), where)
    if out is None:
        out = _empty(x, stream, (T, H, P), _BF16)
    if ht is None and want_ht:
        ht = _empty(x, stream, state, _F32)
    sp = sb = 0
    if scratch is not None or need.value:
        scratch, sp, sb = _scratch(where, dev, scratch, need.value, x, stream)
    code = lib.ssm_fwd(*args, 1 if softplus else 0, cu, cuh, n, T, H, P, G, NS,
                       _dense(where, dev, "h0", h0, _F32, state), _dense(where, dev, "out", out, _BF16, (T, H, P)),
                       _dense(where, dev, "ht", ht, _F32, state), sp, sb, _raw(stream, dev))
    if code:
        _check(code, where)
    return out, ht


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, softplus=True, slots=None, out=None, stream=None):
    """One token of each sequence through the scan: x [B, H, P], dt [B, H], B and
    C [B, G, NS], state fp32 [S, H, NS, P] updated in place; slots as in
    sconv_step.  Returns out bf16 [B, H, P]."""
    where = "ssm_step"
    dev = _device(where, x)
    T, H, P, G, NS, args = _ssm_args(where, dev, x, dt, A, B, C, D, dt_bias)
    if out is None:
        out = _empty(x, stream, (T, H, P), _BF16)
        op = out.data_ptr()
    else:
        op = _dense(where, dev, "out", out, _BF16, (T, H, P))
    S = state.shape[0]
    code = _library().ssm_step(*args, 1 if softplus else 0, _dense(where, dev, "state", state, _F32, (S, H, NS, P)),
                               _dense(where, dev, "slots", slots, _I32, (T,)), T, S, H, P, G, NS, op,
                               _raw(stream, dev))
    if code:
        _check(code, where)
    return out


# ---------------------------------------------------------------------------
# One token of the gated delta rule
# ---------------------------------------------------------------------------
def _delta_step(where, kda, q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream):
    dev = _device(where, q)
    if q.dim() != 3 or v.dim() != 3 or q.shape[2] != 128:
        _fail(where, f"q has shape {tuple(q.shape)} and v {tuple(v.shape)}, expected [batch, heads, 128]")
    heads = q.shape
    B, Hqk, _ = heads
    HV, S = v.shape[1], state.shape[0]
    if kda and Hqk != HV:
        _fail(where, f"q and k have {Hqk} heads and v has {HV}; KDA needs the same count")
    if Hqk < 1 or HV % Hqk:
        _fail(where, f"{HV} value heads do not share {Hqk} q/k heads evenly")
    vals = (B, HV, 128)
    if out is None:
        out = _empty(q, stream, vals, _BF16)
        op = out.data_ptr()
    else:
        op = _dense(where, dev, "out", out, _BF16, vals)
    ptrs = (_dense(where, dev, "q", q, _BF16, heads), _dense(where, dev, "k", k, _BF16, heads),
            _dense(where, dev, "v", v, _BF16, vals), _dense(where, dev, "g", g, _F32, vals if kda else (B, HV)),
            _dense(where, dev, "beta", beta, _BF16 if kda else _F32, (B, HV)),
            _dense(where, dev, "state", state, _F32, (S, HV, 128, 128)),
            _dense(where, dev, "slots", slots, _I32, (B,)), B, S)
    tail = (scale, 1 if qk_l2norm else 0, op, _raw(stream, dev))
    code = _library().kda_step(*ptrs, HV, *tail) if kda else _library().gdn_step(*ptrs, Hqk, HV, *tail)
    if code:
        _check(code, where)
    return out


def kda_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through KDA: q, k, v bf16 [B, H, 128], g fp32
    [B, H, 128], beta bf16 [B, H], state fp32 [S, H, 128, 128] (a forward's ht)
    updated in place; slots as in sconv_step.  Returns out bf16 [B, H, 128]."""
    return _delta_step("kda_step", True, q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream)


def gdn_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through grouped GDN: q, k bf16 [B, Hqk, 128], v
    bf16 [B, HV, 128], g, beta fp32 [B, HV], state fp32 [S, HV, 128, 128]."""
    return _delta_step("gdn_step", False, q, k, v, g, beta, state, scale, slots, out, qk_l2norm, stream)


# ---------------------------------------------------------------------------
# Norms around a block
# ---------------------------------------------------------------------------
def _row_strides(where, dev, name, t, x, shape):
    """(address, outer stride, inner stride) of a row tensor shaped like x: [..., D]
    viewed as [R0, R1, D] with dense rows."""
    if t is None:
        return _NONE3
    if t is not x:
        if t.shape != shape or t.dtype is not x.dtype:
            _fail(where, f"{name} is {t.dtype} {tuple(t.shape)}, expected {x.dtype} {tuple(shape)}")
        _on(where, dev, name, t)
    s = t.stride()
    D = shape[-1]
    if s[-1] != 1 and D > 1:
        _fail(where, f"{name} must have dense rows")
    nd = len(s)
    if nd == 3:
        return t.data_ptr(), s[0], s[1]
    if nd == 2:
        return t.data_ptr(), s[0], D
    if nd == 1:
        return t.data_ptr(), D, D
    if not t.is_contiguous():
        _fail(where, f"{name} has {nd} dimensions and must be contiguous")
    return t.data_ptr(), D * shape[-2], D


def _norm_args(where, dev, x, weight, post_weight, gate, act, residual, res_scale, eps):
    """(shape, D, the library's arguments up to eps)"""
    t, shape = x.dtype, x.shape
    dt = _DTYPE.get(t)
    if dt is None:
        _fail(where, f"x is {t}; bfloat16, float16 and float32 are supported")
    nd = len(shape)
    if nd < 1 or not 1 <= shape[-1] <= 16384:
        _fail(where, f"x has shape {tuple(shape)}; rows of 1 to 16384 elements are supported")
    if act not in _ACT:
        _fail(where, f"act {act!r}, expected 'silu' or 'sigmoid'")
    w = weight if weight is not None else post_weight
    if w is None and residual is None:
        _fail(where, "one of weight, post_weight and residual is needed")
    D = shape[-1]
    R1 = shape[-2] if nd >= 3 else 1
    R0 = x.numel() // (R1 * D) if R1 else 0
    wt = t if w is None else w.dtype
    if wt is not t and wt is not _F32:
        _fail(where, f"weights are {wt}, expected {t} or float32")
    vec = (D,)
    return shape, D, (dt, R0, R1 or 1, D, *_row_strides(where, dev, "x", x, x, shape),
                      *_row_strides(where, dev, "gate", gate, x, shape), _ACT[act],
                      *_row_strides(where, dev, "residual", residual, x, shape), res_scale,
                      _dense(where, dev, "post_weight", post_weight, wt, vec),
                      _dense(where, dev, "weight", weight, wt, vec), _DTYPE[wt], eps)


def norm_workspace_bytes(D: int) -> int:
    """Scratch bytes of norm_bwd for rows of D elements; host only."""
    n = ctypes.c_size_t(0)
    _check(_library().norm_workspace_bytes(D, ctypes.byref(n)), "norm_workspace_bytes")
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
    shape, _, args = _norm_args(where, dev, x, weight, post_weight, gate, act, residual, res_scale, eps)
    t = x.dtype
    hp = yp = 0
    if h is not None:
        hp = _dense(where, dev, "h", h, t, shape)
    elif residual is not None or weight is None:
        h = _empty(x, stream, shape, t)
        hp = h.data_ptr()
    if y is not None:
        yp = _dense(where, dev, "y", y, t, shape)
    elif weight is not None:
        y = _empty(x, stream, shape, t)
        yp = y.data_ptr()
    code = _library().norm_fwd(*args, hp, yp, _raw(stream, dev))
    if code:
        _check(code, where)
    return h, y


def norm_bwd(x, weight=None, post_weight=None, gate=None, act="silu", residual=None, res_scale=1.0, eps=1e-6, dh=None,
             dy=None, scratch=None, grads=None, stream=None):
    """Gradients of norm_fwd from dh and dy (the gradients of h and y; either may
    be None).  Returns a dict with dx and, for the arguments given, dgate,
    dresidual, dweight and dpost_weight (fp32); `grads` may bring preallocated
    tensors.  Where u = x and res_scale = 1, dx and dresidual are one tensor."""
    where = "norm_bwd"
    dev = _device(where, x)
    shape, D, args = _norm_args(where, dev, x, weight, post_weight, gate, act, residual, res_scale, eps)
    t = x.dtype
    if dh is None and dy is None:
        _fail(where, "one of dh and dy is needed")
    if dy is not None and weight is None:
        _fail(where, "dy without weight")
    got = dict(grads or {})
    same = residual is not None and post_weight is None and gate is None and res_scale == 1.0 and not grads
    for name, given in (("dx", x), ("dgate", gate), ("dresidual", residual)):
        if given is not None and name not in got:
            got[name] = got["dx"] if same and name == "dresidual" else _empty(x, stream, shape, t)
    for name, given in (("dweight", weight), ("dpost_weight", post_weight)):
        if given is not None and name not in got:
            got[name] = _empty(x, stream, (D,), _F32)
    scratch, sp, sb = _scratch(where, dev, scratch, norm_workspace_bytes(D), x, stream)
    code = _library().norm_bwd(*args, *_row_strides(where, dev, "dh", dh, x, shape),
                               *_row_strides(where, dev, "dy", dy, x, shape),
                               _dense(where, dev, "dx", got.get("dx"), t, shape),
                               _dense(where, dev, "dgate", got.get("dgate"), t, shape),
                               0 if same else _dense(where, dev, "dresidual", got.get("dresidual"), t, shape),
                               _dense(where, dev, "dweight", got.get("dweight"), _F32, (D,)),
                               _dense(where, dev, "dpost_weight", got.get("dpost_weight"), _F32, (D,)), sp, sb,
                               _raw(stream, dev))
    if code:
        _check(code, where)
    return got
