"""The operators around the gated delta rule: the short causal convolution, the
selective state space scan, the single-token forms and the norms around a
block (``include/gdr.h``).  Thin names over the compiled binding
(csrc/gdr_binding.cpp), re-exported by the package; all arguments are checked for device,
type, shape and layout before the library is called, and a check that fails
raises ``ValueError`` with nothing enqueued.

Outputs and workspaces are allocated on the stream the call runs on: `stream`,
or the current one.  Inputs that belong to another stream are the caller's to order
before the call and to keep until it has run (``Tensor.record_stream``).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

import numpy as np
import torch

from . import _check, build, load

__all__ = ("sconv_workspace_bytes", "sconv_fwd", "sconv_bwd", "sconv_step", "ssm_workspace_bytes", "ssm_fwd", "ssm_step",
           "kda_step", "gdn_step", "norm_workspace_bytes", "norm_fwd", "norm_bwd")


def _load_binding():
    load()
    path = build.binding_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{os.path.basename(path)} not found at {path}; build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    loader = importlib.machinery.ExtensionFileLoader("_gdr_ops", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_gdr_ops", loader))
    loader.exec_module(module)
    module.set_check(_check)
    return module


_binding = _load_binding()


def _on(stream, call, *args):
    """The call on a stream of the caller's, where its tensors are allocated too."""
    with torch.cuda.stream(stream):
        return call(*args)


def _host(cu_seqlens_host):
    """A C-contiguous int32 array."""
    h = cu_seqlens_host
    if type(h) is np.ndarray and h.dtype == np.int32 and h.flags.c_contiguous:
        return h
    if hasattr(h, "detach"):
        h = h.detach().cpu().numpy()
    return np.ascontiguousarray(h, dtype=np.int32)


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
    if stream is not None:
        return _on(stream, _binding.sconv_fwd, x, weight, bias, cu_seqlens, _host(cu_seqlens_host), s0, silu, out,
                   st, want_st)
    return _binding.sconv_fwd(x, weight, bias, cu_seqlens, _host(cu_seqlens_host), s0, silu, out, st, want_st)


def sconv_bwd(x, weight, bias, cu_seqlens, cu_seqlens_host, dout, s0=None, dst=None, want_ds0=False, silu=True,
              scratch=None, grads=None, stream=None):
    """Gradients of sconv_fwd from dout [T, C] (and dst, the gradient of st).
    Returns a dict with dx, dweight (fp32), dbias (fp32, None without a bias)
    and, when wanted, ds0; `grads` may bring preallocated tensors."""
    if stream is not None:
        return _on(stream, _binding.sconv_bwd, x, weight, bias, cu_seqlens, _host(cu_seqlens_host), dout, s0, dst,
                   want_ds0, silu, scratch, grads)
    return _binding.sconv_bwd(x, weight, bias, cu_seqlens, _host(cu_seqlens_host), dout, s0, dst, want_ds0, silu,
                              scratch, grads)


def sconv_step(x, weight, bias, state, slots=None, silu=True, out=None, stream=None):
    """One token of each sequence: x [B, C], state [S, W-1, C] updated in place,
    slots int32 [B] (None: row b uses state b; a slot outside [0, S) makes the
    row inactive).  Returns out [B, C]."""
    if stream is not None:
        return _on(stream, _binding.sconv_step, x, weight, bias, state, slots, silu, out)
    return _binding.sconv_step(x, weight, bias, state, slots, silu, out)


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
    (out bf16 [T, H, P], ht fp32 [N, H, NS, P] or None).

    P and NS go up to 256.  Chunks on the tensor cores need P and NS in multiples of
    8, NS <= 128 and rows on 16-byte boundaries; other sizes go token by token, about
    25 times slower on a long prompt."""
    if stream is not None:
        return _on(stream, _binding.ssm_fwd, x, dt, A, B, C, D, dt_bias, softplus, cu_seqlens,
                   _host(cu_seqlens_host), h0, out, ht, want_ht, scratch)
    return _binding.ssm_fwd(x, dt, A, B, C, D, dt_bias, softplus, cu_seqlens, _host(cu_seqlens_host), h0, out, ht,
                            want_ht, scratch)


def ssm_step(x, dt, A, B, C, state, D=None, dt_bias=None, softplus=True, slots=None, out=None, stream=None):
    """One token of each sequence through the scan: x [B, H, P], dt [B, H], B and
    C [B, G, NS], state fp32 [S, H, NS, P] updated in place; slots as in
    sconv_step.  Returns out bf16 [B, H, P]."""
    if stream is not None:
        return _on(stream, _binding.ssm_step, x, dt, A, B, C, D, dt_bias, softplus, state, slots, out)
    return _binding.ssm_step(x, dt, A, B, C, D, dt_bias, softplus, state, slots, out)


def kda_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through KDA: q, k, v bf16 [B, H, 128], g fp32
    [B, H, 128], beta bf16 [B, H], state fp32 [S, H, 128, 128] (a forward's ht)
    updated in place; slots as in sconv_step.  Returns out bf16 [B, H, 128]."""
    if stream is not None:
        return _on(stream, _binding.kda_step, q, k, v, g, beta, state, scale, slots, out, qk_l2norm)
    return _binding.kda_step(q, k, v, g, beta, state, scale, slots, out, qk_l2norm)


def gdn_step(q, k, v, g, beta, state, scale, slots=None, out=None, qk_l2norm=False, stream=None):
    """One token of each sequence through grouped GDN: q, k bf16 [B, Hqk, 128], v
    bf16 [B, HV, 128], g, beta fp32 [B, HV], state fp32 [S, HV, 128, 128]."""
    if stream is not None:
        return _on(stream, _binding.gdn_step, q, k, v, g, beta, state, scale, slots, out, qk_l2norm)
    return _binding.gdn_step(q, k, v, g, beta, state, scale, slots, out, qk_l2norm)


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
    if stream is not None:
        return _on(stream, _binding.norm_fwd, x, weight, post_weight, gate, act, residual, res_scale, eps, h, y)
    return _binding.norm_fwd(x, weight, post_weight, gate, act, residual, res_scale, eps, h, y)


def norm_bwd(x, weight=None, post_weight=None, gate=None, act="silu", residual=None, res_scale=1.0, eps=1e-6, dh=None,
             dy=None, scratch=None, grads=None, stream=None):
    """Gradients of norm_fwd from dh and dy (the gradients of h and y; either may
    be None).  Returns a dict with dx and, for the arguments given, dgate,
    dresidual, dweight and dpost_weight (fp32); `grads` may bring preallocated
    tensors.  Where u = x and res_scale = 1, dx and dresidual are one tensor."""
    if stream is not None:
        return _on(stream, _binding.norm_bwd, x, weight, post_weight, gate, act, residual, res_scale, eps, dh, dy,
                   scratch, grads)
    return _binding.norm_bwd(x, weight, post_weight, gate, act, residual, res_scale, eps, dh, dy, scratch, grads)
