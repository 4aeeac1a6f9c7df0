"""Plain 64-bit references of the operators around the recurrence, for the tests:
token by token (or document by document) from the definitions in include/gdr.h,
on whatever device the inputs are on; gradients by torch autograd in FP64.

Tolerances (relative L2 over a tensor), from the formats:
* an output rounded once to n significand bits is off by at most 2^-n of each
  element: bf16 (8 bits with the implicit one) 2^-8 at worst per element and
  2^-8 / (2 sqrt 3) ~ 1.1e-3 to 1.95e-3 in the mean over a binade; 2.5e-3 leaves
  room for the FP32 (or split-BF16, 16 bits) arithmetic before the rounding;
* fp16, three bits more: 3.5e-4;
* FP32 outputs of sums: 1e-5 (unit roundoff 6e-8, exponentials to 2 ulp, sums of
  up to a few thousand terms; the scan's BF16 pairs carry 16 bits, 2^-17 = 7.6e-6
  at worst per term and less in the mean).
"""
import torch

TOL = {torch.bfloat16: 2.5e-3, torch.float16: 3.5e-4, torch.float32: 1e-5}


def rel(a, b):
    a, b = a.detach().double(), b.detach().double().to(a.device)
    n = float(b.norm())
    d = float((a - b).norm())
    return d / n if n else d


def check(got, ref, what, tol=None):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got.double()).all(), f"{what}: not finite"
    e, t = rel(got, ref), TOL[got.dtype] if tol is None else tol
    assert e <= t, f"{what}: relative error {e:.3e} > {t:.1e}"
    return e


def cu_of(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def conv(x, w, b, lengths, s0, silu):
    """(out, end states); x, w, b, s0 FP64."""
    K = w.shape[1] - 1
    outs, ends, at = [], [], 0
    for i, n in enumerate(lengths):
        pre = s0[i] if s0 is not None else x.new_zeros(K, x.shape[1])
        xx = torch.cat([pre, x[at:at + n]])
        z = sum(xx[j:j + n] * w[:, j] for j in range(K + 1))
        z = z if b is None else z + b
        outs.append(z * torch.sigmoid(z) if silu else z)
        ends.append(xx[n:])
        at += n
    return torch.cat(outs), torch.stack(ends)


def scan(x, dt, A, B, C, D, lengths, h0):
    """(out, end states) of S_t = exp(dt A) S + dt B x^T, out = S^T C + D x; FP64, dt activated."""
    T, H, P = x.shape
    G, N = B.shape[1:]
    Bh, Ch = (t.repeat_interleave(H // G, 1) for t in (B, C))
    out, ends, at = torch.empty_like(x), [], 0
    for i, n in enumerate(lengths):
        S = h0[i].clone() if h0 is not None else x.new_zeros(H, N, P)
        for t in range(at, at + n):
            S = torch.exp(dt[t] * A)[:, None, None] * S + (dt[t][:, None] * Bh[t])[:, :, None] * x[t][:, None, :]
            out[t] = torch.einsum("hnp,hn->hp", S, Ch[t])
        ends.append(S)
        at += n
    return out if D is None else out + D[:, None] * x, torch.stack(ends)


def delta(q, k, v, g, beta, S, scale, l2):
    """(out, new states) of one token; q, k already repeated to the value heads, S [B, H, 128, 128]."""
    if l2:
        q, k = (t * (t.square().sum(-1, keepdim=True) + 1e-6).rsqrt() for t in (q, k))
    a = torch.exp(g)
    S = S * (a[..., None] if a.dim() == 3 else a[..., None, None])
    d = beta[..., None] * (v - torch.einsum("bhkv,bhk->bhv", S, k))
    S = S + k[..., None] * d[..., None, :]
    return scale * torch.einsum("bhkv,bhk->bhv", S, q), S


def norms(x, w, w_post, z, act, r, alpha, eps):
    """(h, y); y None without w."""
    u = x
    if w_post is not None:
        u = u * (u.square().mean(-1, keepdim=True) + eps).rsqrt() * w_post
    if z is not None:
        u = u * torch.sigmoid(z) * (z if act == "silu" else 1)
    h = r + alpha * u if r is not None else u
    y = h * (h.square().mean(-1, keepdim=True) + eps).rsqrt() * w if w is not None else None
    return h, y
