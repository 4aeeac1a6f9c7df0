"""Plain 64-bit references of the attention layer's operators (layer norm, rotary
positions, attention over packed documents), from the definitions in include/gdr.h;
gradients by torch autograd in FP64.

Tolerances (relative L2 over a tensor), from the formats.  Rounding to bf16 is off by
at most 2^-8 of an element, 2^-8 / sqrt(3) of its binade's lower end in the mean: 1.66e-3
over a tensor.  The tensor cores take two more factors in bf16:
* attention's probabilities P, so that out = P v and dv = P^T dout are off by 1.66e-3
  (the terms' errors are independent) and by their own rounding: 2.35e-3 together;
* dS = P (dP - delta), of which delta = dout . out comes from the rounded out (2.35e-3 of
  |out| <= |v|): dq and dk are off by sqrt(1.66^2 + 1.66^2 + 2.35^2) 1e-3 = 3.3e-3.
A fifth is left for the spread of small tensors.  lse is FP32: products of up to 256
terms in FP32 sums, exponentials to 2^-22, against values of order one and more.
"""
import math

import torch

TOL_OUT, TOL_GRAD, TOL_LSE = 2.9e-3, 4e-3, 1e-5


def attention(q, k, v, lens_q, lens_k, scale, causal, window):
    """(out [T, H, D], lse [H, T]); q, k, v FP64."""
    G, outs, lses, a, b = q.shape[1] // k.shape[1], [], [], 0, 0
    for n, m in zip(lens_q, lens_k):
        Q = q[a:a + n].transpose(0, 1)
        K, V = (t[b:b + m].repeat_interleave(G, 1).transpose(0, 1) for t in (k, v))
        s = scale * Q @ K.transpose(-1, -2)  # [H, n, m]
        if causal:
            gap = torch.arange(n, device=q.device)[:, None] + (m - n) - torch.arange(m, device=q.device)
            s = s.masked_fill((gap < 0) | (gap >= window) if window else gap < 0, -math.inf)
        none = (s == -math.inf).all(-1, keepdim=True)
        lse = torch.logsumexp(torch.where(none, 0.0, s), -1) if m else s.new_zeros(s.shape[:2])
        p = torch.where(none, 0.0, torch.exp(s - lse[..., None]))
        outs.append((p @ V).transpose(0, 1))
        lses.append(torch.where(none[..., 0], -math.inf, lse))
        a, b = a + n, b + m
    return torch.cat(outs), torch.cat(lses, 1)


def layer_norm(x, w, b, r, alpha, eps):
    """(h, y)"""
    h = x if r is None else r + alpha * x
    d = h - h.mean(-1, keepdim=True)
    y = d / torch.sqrt(d.square().mean(-1, keepdim=True) + eps)
    y = y if w is None else y * w
    return h, y if b is None else y + b


def rotate(x, positions, freqs, interleaved, amplitude):
    R = 2 * freqs.shape[0]
    angle = positions.double()[:, None] * freqs.double()
    c, s = (amplitude * f(angle)[:, None] for f in (torch.cos, torch.sin))
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    p, q = a * c - b * s, b * c + a * s
    out = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([out, x[..., R:]], -1)
