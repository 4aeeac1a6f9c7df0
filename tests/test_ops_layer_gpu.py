"""The attention layer's operators (layer norm, rotary positions, attention over packed
documents) on the GPU against the plain FP64 references of layer_ref.py."""
import math

import pytest
import torch

import layer_ref as ref
from layer_ref import TOL_GRAD, TOL_LSE, TOL_OUT
from ops_ref import check, cu_of, rel

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def gdr():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import gated_delta_rule_varlen_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def full(shape, dtype):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


def pack(lengths):
    cu = cu_of(lengths)
    return torch.tensor(cu, dtype=torch.int32, device="cuda"), cu


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
LNORM = [
    # shape, dtype, weight, bias, residual, fp32 weights, element offset of the inputs, extra elements a row
    ((1, 2048), BF16, True, True, True, False, 0, 0), ((37, 128), BF16, True, False, False, False, 0, 0),
    ((5, 3, 64), F16, True, True, True, True, 0, 8), ((300, 1021), F32, True, True, True, False, 0, 0),
    ((9, 1000), BF16, False, False, True, False, 0, 0), ((33, 77), BF16, True, True, True, False, 1, 3),
    ((7, 1), F32, True, True, False, False, 0, 0), ((6, 2), F32, True, True, True, False, 0, 0),
    ((4, 3), F16, True, True, False, False, 0, 0), ((3, 16384), BF16, True, True, True, True, 0, 0),
    ((11, 5000), F32, True, True, False, False, 0, 0), ((2, 8200), F16, True, False, True, False, 0, 0),
    ((2, 9001), BF16, True, True, True, False, 1, 1), ((2000, 16), BF16, True, True, False, False, 0, 0),
    ((1000, 24), F32, False, True, True, False, 0, 0), ((8191, 136), F16, True, True, True, False, 0, 0),
    ((3, 16383), F32, True, True, True, False, 0, 0), ((50, 4, 520), BF16, True, True, True, False, 0, 16),
]


def rows_of(t, offset, pad):
    """The same values in wider rows that start `offset` elements in."""
    if not (offset or pad):
        return t
    wide = torch.full((*t.shape[:-1], t.shape[-1] + pad + offset), 7.0, dtype=t.dtype, device=t.device)
    view = wide[..., offset:offset + t.shape[-1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("shape,dtype,weight,bias,residual,wf32,offset,pad", LNORM)
def test_lnorm_forward_and_gradients(gdr, shape, dtype, weight, bias, residual, wf32, offset, pad):
    g, D, wt = gen(shape[0] + shape[-1]), shape[-1], F32 if wf32 else dtype
    x = (randn(g, *shape) + 3).to(dtype)
    r = randn(g, *shape).mul(2).to(dtype) if residual else None
    w = randn(g, D).mul(0.3).add(1).to(wt) if weight else None
    b = randn(g, D).to(wt) if bias else None
    dy, dh = (randn(g, *shape, dtype=dtype) for _ in range(2))
    alpha, eps = (0.5, 1e-5) if residual else (1.0, 1e-5)
    xs, rs, dys, dhs = (None if t is None else rows_of(t, offset, pad) for t in (x, r, dy, dh))
    h, y = gdr.lnorm_fwd(xs, w, b, residual=rs, res_scale=alpha, eps=eps, y=full(shape, dtype))
    leaves = [None if t is None else t.double().requires_grad_() for t in (x, w, b, r)]
    rh, ry = ref.layer_norm(*leaves, alpha, eps)
    if D > 2:  # (of one element y is the bias, of two the sign of their difference)
        check(y, ry, "y")
    assert (y.double() - ry.detach()).abs().max() <= 2 ** -7 * max(1.0, float(ry.detach().abs().max()))
    if residual:
        check(h, rh, "h")
    else:
        assert h is None
    # the sums' FP32 rounding beside a gradient that cancels: of rows of one or two elements
    # dx is (nearly) zero
    got = gdr.lnorm_bwd(xs, w, b, residual=rs, res_scale=alpha, eps=eps, dh=dhs, dy=dys, grads={"dx": full(shape, dtype)})
    total = (ry * dy.double()).sum() + (rh * dh.double()).sum()
    want = [t for t in leaves if t is not None]
    grads = dict(zip([n for n, t in zip(("dx", "dweight", "dbias", "dresidual"), leaves) if t is not None],
                     torch.autograd.grad(total, want)))
    assert set(grads) <= {k for k, t in got.items() if t is not None}
    for name, t in grads.items():
        if D == 1 and name == "dweight":
            assert float(got[name].abs().max()) <= 1e-3  # n = 0
        else:
            check(got[name], t, name)
    again = gdr.lnorm_bwd(xs, w, b, residual=rs, res_scale=alpha, eps=eps, dh=dhs, dy=dys)
    for name in grads:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("D", [2, 3, 64, 1000])
def test_lnorm_gradient_without_dh(gdr, D):
    # alone, what cancels in r (dn - mean - n mean(dn n)) is not hidden behind dh
    g = gen(D)
    x, w, dy = randn(g, 40, D) * 3, randn(g, D) + 1, randn(g, 40, D)
    leaf = x.double().requires_grad_()
    want, = torch.autograd.grad((ref.layer_norm(leaf, w.double(), None, None, 1.0, 1e-5)[1] * dy.double()).sum(), leaf)
    got = gdr.lnorm_bwd(x, w, dy=dy)["dx"]
    # FP32: dn and its mean are off by 2^-24 of |dn|, of which n takes the most part in short rows
    if D == 2:
        near = (x[:, 0] - x[:, 1]).abs() > 0.3
        assert rel(got[near], want[near]) <= 1e-5 and rel(got, want) <= 1e-3
    else:
        assert rel(got, want) <= 2e-5


def test_lnorm_far_from_zero(gdr):
    # a mean of 1000 beside a spread of 1: squares of the rows themselves would keep 4 bits of it
    g = gen(5)
    x = randn(g, 64, 4096) + 1000
    _, y = gdr.lnorm_fwd(x)
    # the inputs are exact, the mean is off by 2^-24 1000 at most: 6e-5 of the spread
    assert (y.double() - ref.layer_norm(x.double(), None, None, None, 1.0, 1e-5)[1]).abs().max() <= 2e-4


def test_lnorm_in_place_and_refusals(gdr):
    g = gen(3)
    x, r, w = randn(g, 20, 256, dtype=BF16), randn(g, 20, 256, dtype=BF16), randn(g, 256, dtype=BF16)
    h, y = gdr.lnorm_fwd(x, w, residual=r)
    r2, x2 = r.clone(), x.clone()
    gdr.lnorm_fwd(x2, w, residual=r2, h=r2, y=x2)
    assert torch.equal(r2, h) and torch.equal(x2, y)
    for bad in (lambda: gdr.lnorm_fwd(x, w[:100]), lambda: gdr.lnorm_fwd(x, w, residual=r[:5]), lambda: gdr.lnorm_fwd(x.long()),
                lambda: gdr.lnorm_fwd(x, w, bias=w.float()), lambda: gdr.lnorm_bwd(x, w, dh=x), lambda: gdr.lnorm_fwd(x.t()),
                lambda: gdr.lnorm_fwd(x, w, y=r[:3]), lambda: gdr.lnorm_bwd(x, w, dy=r, scratch=torch.empty(16, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    e = gdr.lnorm_bwd(x[:0], w, w, dy=x[:0])
    assert e["dx"].shape == (0, 256) and float(e["dweight"].abs().max()) == 0 and float(e["dbias"].abs().max()) == 0


# ---------------------------------------------------------------------------
# Rotary positions
# ---------------------------------------------------------------------------
ROPE = [
    # T, H, HK, D, R, interleaved, dtype, extra elements a token, element offset
    (1, 16, 4, 128, 128, False, BF16, 0, 0), (37, 4, 1, 128, 64, True, F16, 128, 0), (300, 3, 3, 80, 40, False, BF16, 0, 0),
    (65, 5, 1, 96, 96, True, F32, 0, 0), (50, 2, 2, 64, 64, False, F32, 1, 1), (33, 2, 1, 63, 34, True, BF16, 1, 1),
    (33, 2, 1, 63, 34, False, F16, 0, 0), (7, 1, 1, 2, 2, True, F32, 0, 0), (9, 8, 0, 256, 0, False, BF16, 0, 0),
    (2000, 32, 8, 128, 128, False, BF16, 256, 0), (700, 40, 8, 64, 16, True, BF16, 0, 0), (130, 6, 2, 68, 68, True, F16, 2, 2),
]


@pytest.mark.parametrize("T,H,HK,D,R,interleaved,dtype,pad,offset", ROPE)
def test_rope_and_its_gradient(gdr, T, H, HK, D, R, interleaved, dtype, pad, offset):
    g = gen(T + D)
    wide = randn(g, T, (H + HK) * D + pad + offset, dtype=dtype)
    q = wide[:, offset:offset + H * D].unflatten(1, (H, D))
    k = wide[:, offset + H * D:offset + (H + HK) * D].unflatten(1, (HK, D)) if HK else None
    f = gdr.rope_frequencies(R, base=500.0)
    pos = torch.randint(-5000, 1 << 30, (T,), generator=g, device="cuda", dtype=torch.int32)
    got = gdr.rope_fwd(q, k, f, positions=pos, interleaved=interleaved, amplitude=1.25)
    for x, y in zip((q, k), got):
        if x is None:
            assert y is None
            continue
        check(y, ref.rotate(x.double(), pos, f, interleaved, 1.25), "turned")
        assert torch.equal(y[..., R:], x[..., R:]), "the rest is copied"
    # the same in place, positions of 64 bits; back is the transpose: <rope q, z> = <q, rope_bwd z>
    z = randn(g, T, H, D, dtype=dtype)
    back, _ = gdr.rope_bwd(z, None, f, positions=pos.long(), interleaved=interleaved, amplitude=1.25)
    leaf = q.double().requires_grad_()
    want, = torch.autograd.grad((ref.rotate(leaf, pos, f, interleaved, 1.25) * z.double()).sum(), leaf)
    check(back, want, "back")
    before = wide.clone()
    gdr.rope_fwd(q, k, f, positions=pos.long(), interleaved=interleaved, amplitude=1.25, q_out=q, k_out=k)
    assert torch.equal(q, got[0]) and (k is None or torch.equal(k, got[1]))
    assert torch.equal(wide[:, :offset], before[:, :offset])
    assert torch.equal(wide[:, offset + (H + HK) * D:], before[:, offset + (H + HK) * D:])


def test_rope_counts_from_each_document(gdr):
    g, lengths = gen(1), [3, 0, 1, 70, 0, 5]
    cu, _ = pack(lengths)
    T = sum(lengths)
    q = randn(g, T, 2, 64)
    f = gdr.rope_frequencies(64)
    pos = torch.cat([torch.arange(n) for n in lengths]).cuda().int()
    a, _ = gdr.rope_fwd(q, None, f, cu_seqlens=cu)
    b, _ = gdr.rope_fwd(q, None, f, positions=pos)
    assert torch.equal(a, b)


def test_rope_far_positions_keep_their_angle(gdr):
    # FP32 products of position and frequency would be off by 2^31 2^-24 = 128 radians
    pos = torch.tensor([0, 1, 2**20 + 1, 2**31 - 1, -(2**31), -1, 123456789], dtype=torch.int32, device="cuda")
    f = gdr.rope_frequencies(128, base=1e6)
    q = torch.zeros(7, 1, 128, device="cuda")
    q[..., :64] = 1
    y, _ = gdr.rope_fwd(q, None, f, positions=pos)
    want = ref.rotate(q.double(), pos, f, False, 1.0)
    # the FP64 product's own rounding: 2^31 2^-53 = 2.4e-7; the fraction's top 32 bits as FP32 2^-25 turns
    assert (y.double() - want).abs().max() <= 8e-7
    f2 = torch.tensor([0.0, 1e-30, 1.0, 3.0, 100.0, -0.5, 2.0**-126, 2.0**-140], device="cuda")
    q = randn(gen(2), 7, 1, 16)
    y, _ = gdr.rope_fwd(q, None, f2, positions=pos // 64, interleaved=True)
    assert (y.double() - ref.rotate(q.double(), pos // 64, f2, True, 1.0)).abs().max() <= 2e-5


def test_rope_refusals(gdr):
    q, k = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, 1, 64, device="cuda")
    f, pos = gdr.rope_frequencies(64), torch.arange(4, device="cuda", dtype=torch.int32)
    gdr.rope_fwd(q, k, f, positions=pos)
    for bad in (lambda: gdr.rope_fwd(q, k, f), lambda: gdr.rope_fwd(None, None, f, positions=pos), lambda: gdr.rope_fwd(q, k[:3], f, positions=pos),
                lambda: gdr.rope_fwd(q, k.half(), f, positions=pos), lambda: gdr.rope_fwd(q, k, f[:, None], positions=pos),
                lambda: gdr.rope_fwd(q, k, torch.zeros(33, device="cuda"), positions=pos), lambda: gdr.rope_fwd(q, k, f.double(), positions=pos),
                lambda: gdr.rope_fwd(q, k, f, positions=pos[:3]), lambda: gdr.rope_fwd(q, k, f, positions=pos.float()),
                lambda: gdr.rope_fwd(q, k, f, positions=pos, q_out=q[:, :1]), lambda: gdr.rope_fwd(q, None, f, positions=pos, k_out=k),
                lambda: gdr.rope_fwd(q.transpose(1, 2), None, f, positions=pos), lambda: gdr.rope_fwd(q[0], None, f, positions=pos)):
        with pytest.raises(ValueError):
            bad()
    y, _ = gdr.rope_fwd(q[:0], None, f, positions=pos[:0])
    assert y.shape == (0, 2, 64)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
RAGGED = [1, 63, 64, 0, 65, 129, 300]
ATTN = [
    # queries, keys (None: the same), H, HK, D, causal, window, layout
    (RAGGED, None, 4, 4, 128, True, 0, "fused"), (RAGGED, None, 4, 4, 64, False, 0, "fused"),
    ([1], None, 1, 1, 128, True, 0, "dense"), ([2, 1], None, 2, 1, 64, True, 0, "dense"),
    ([128, 127, 256, 257], None, 6, 2, 128, True, 0, "fused"), ([500], None, 8, 1, 128, True, 0, "heads"),
    ([383, 5, 1000], None, 4, 2, 128, True, 128, "fused"), ([777], None, 2, 2, 64, True, 1, "dense"),
    ([900], None, 2, 1, 128, True, 200, "dense"), ([640], None, 5, 5, 80, True, 0, "fused"),
    ([333, 20], None, 3, 1, 96, False, 0, "dense"), ([200], None, 2, 2, 40, True, 33, "dense"),
    ([130, 9], None, 2, 1, 8, True, 0, "dense"),
    # other keys: prompts behind cached keys, single tokens, fewer keys than queries, none
    ([1] * 9, [1, 2, 127, 128, 129, 1000, 300, 0, 77], 8, 2, 128, True, 0, "dense"),
    ([1] * 3, [5000, 3, 129], 8, 8, 64, True, 0, "dense"), ([1] * 2, [5000, 3000], 12, 4, 128, True, 1000, "dense"),
    ([7, 130, 0, 4], [900, 131, 50, 4], 6, 2, 128, True, 0, "dense"), ([300, 40], [200, 0], 4, 2, 128, True, 0, "dense"),
    ([300, 129, 1], [170, 128, 0], 4, 2, 64, True, 64, "dense"), ([50, 260], [333, 1], 4, 4, 128, False, 0, "dense"),
    ([2, 3, 1], [600, 258, 4000], 16, 2, 128, True, 0, "dense"),
    # shapes of no tile: odd dimensions, rows on no 16 bytes, wide heads
    ([70, 3, 0, 129], None, 4, 2, 33, True, 0, "dense"), ([100, 28], None, 2, 2, 128, True, 0, "odd"),
    ([65, 30], None, 2, 1, 256, True, 0, "dense"), ([40, 7], [80, 3], 2, 1, 130, True, 20, "dense"), ([20], None, 2, 2, 1, False, 0, "dense"),
]


def heads(g, T, H, HK, D, layout, TK):
    if layout == "dense":
        return randn(g, T, H, D, dtype=BF16), randn(g, TK, HK, D, dtype=BF16), randn(g, TK, HK, D, dtype=BF16)
    if layout == "heads":  # heads outermost
        return tuple(randn(g, h, t, D, dtype=BF16).transpose(0, 1) for h, t in ((H, T), (HK, TK), (HK, TK)))
    wide = randn(g, T, (H + 2 * HK) * D + (1 if layout == "odd" else 24), dtype=BF16)
    at = 1 if layout == "odd" else 16
    return tuple(wide[:, at + a * D:at + b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))


def compare(got, want, tol, what):
    assert got.shape == want.shape, what
    bad = ~torch.isfinite(want)
    assert torch.equal(got.double()[bad], want[bad]), what
    assert torch.isfinite(got[~bad].double()).all(), f"{what}: not finite"
    e = rel(got[~bad], want[~bad])
    assert e <= tol, f"{what}: relative error {e:.3e} > {tol:.1e}"


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window,layout", ATTN)
def test_attention_forward_and_gradients(gdr, lq, lk, H, HK, D, causal, window, layout):
    g, keys = gen(sum(lq) + D), lk or lq
    T, TK = sum(lq), sum(keys)
    q, k, v = heads(g, T, H, HK, D, layout, TK)
    dout = randn(g, T, H, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack(lq), pack(lk) if lk else (None, None)
    args = dict(causal=causal, window=window, cu_keys=cuk, cu_keys_host=cukh)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    ro, rl = ref.attention(*leaves, lq, keys, D ** -0.5, causal, window)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, out=full((T, H, D), BF16), lse=full((H, T), F32), **args)
    compare(lse, rl.detach(), TOL_LSE, "lse")
    compare(out, ro.detach(), TOL_OUT, "out")
    rg = torch.autograd.grad((ro * dout.double()).sum(), leaves)
    grads = {"dq": full((T, H, D), BF16), "dk": full((TK, HK, D), BF16), "dv": full((TK, HK, D), BF16)}
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, grads=grads, **args)
    # a gradient that is zero, or nothing but what cancels (rows that see one key: dS = 0), is
    # compared with the size of its terms: |dS| |k| of one term, 2^-8 of it
    terms = 2 ** -8 * D ** 0.5
    for name, r in zip(("dq", "dk", "dv"), rg):
        t = got[name].double()
        assert torch.isfinite(t).all(), f"{name}: not finite"
        off, size = float((t - r).norm()), float(r.norm())
        assert off <= TOL_GRAD * size or (off / max(1, t.numel()) ** 0.5) <= TOL_GRAD * terms, f"{name}: {off:.3e} of {size:.3e}"
    again = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, **args)
    out2, lse2 = gdr.attn_fwd(q, k, v, cu, cuh, **args)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    for name in got:
        assert torch.equal(got[name], again[name]), name


@pytest.mark.parametrize("D,H,HK", [(64, 2, 1), (128, 3, 3), (36, 2, 2)])
def test_attention_gradients_by_differences(gdr, D, H, HK):
    # along a direction large enough for bf16 steps: the loss is linear in v, and its curvature
    # in q and k is what the symmetric difference drops
    g, lens = gen(D), [40, 150]
    T = sum(lens)
    cu, cuh = pack(lens)
    x = dict(zip("qkv", heads(g, T, H, HK, D, "dense", T)))
    dout = randn(g, T, H, D, dtype=BF16)

    def loss(a):
        # through the FP64 reference, so that only the gradient is the library's
        return float((ref.attention(a["q"], a["k"], a["v"], lens, lens, D ** -0.5, True, 0)[0] * dout.double()).sum())

    out, lse = gdr.attn_fwd(x["q"], x["k"], x["v"], cu, cuh)
    got = gdr.attn_bwd(x["q"], x["k"], x["v"], out, lse, dout, cu, cuh)
    for name in "qkv":
        u = randn(g, *x[name].shape).double()
        base = {n: t.double() for n, t in x.items()}
        up, down = ({**base, name: base[name] + s * 1e-4 * u} for s in (1, -1))
        diff = (loss(up) - loss(down)) / 2e-4
        grad = got["d" + name].double()
        inner = float((grad * u).sum())
        # the gradient's error of TOL_GRAD |grad| against a random direction: three sigmas
        assert abs(diff - inner) <= 3 * TOL_GRAD * float(grad.norm()) + 1e-5 * abs(diff), (name, diff, inner)


def test_attention_scores_far_apart(gdr):
    # scores between -1000 and 1000: maxima that grow along the keys, probabilities that vanish
    g, D = gen(8), 64
    q, k, v = heads(g, 700, 2, 2, D, "dense", 700)
    k = (k.float() * torch.linspace(0.1, 30, 700, device="cuda")[:, None, None]).to(BF16)
    cu, cuh = pack([700])
    for scale in (1.0, 30.0, 1e-3):
        out, lse = gdr.attn_fwd(q, k, v, cu, cuh, scale=scale)
        ro, rl = ref.attention(q.double(), k.double(), v.double(), [700], [700], scale, True, 0)
        # a score is off by 2^-22 of the sum of its terms' sizes, and e^ of it by as much
        off = scale * float((q.double().abs().amax() * k.double().abs().amax() * D)) * 2 ** -22
        assert (lse.double() - rl).abs().max() <= off + 1e-5
        if off < 1e-3:
            compare(out, ro, TOL_OUT, "out")
        assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("bad", [NAN, float("inf"), -float("inf")])
def test_attention_keeps_documents_apart(gdr, bad):
    # tiles reach over a document's end: what is not finite in the next one stays there
    g, lens, D = gen(4), [100, 60, 200, 1, 130], 128
    T = sum(lens)
    cu, cuh = pack(lens)
    q, k, v = heads(g, T, 2, 1, D, "dense", T)
    dout = randn(g, T, 2, D, dtype=BF16)
    clean = gdr.attn_fwd(q, k, v, cu, cuh)
    cleang = gdr.attn_bwd(q, k, v, *clean, dout, cu, cuh)
    q2, k2, v2, d2 = (t.clone() for t in (q, k, v, dout))
    for t in (q2, k2, v2, d2):
        t[100:160] = bad
        t[361:] = bad
    got = gdr.attn_fwd(q2, k2, v2, cu, cuh)
    grads = gdr.attn_bwd(q2, k2, v2, *got, d2, cu, cuh)
    for rows in (slice(0, 100), slice(160, 361)):
        assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][:, rows], clean[1][:, rows])
        for n in cleang:
            assert torch.equal(grads[n][rows], cleang[n][rows]), n


def test_attention_of_scores_that_are_not_numbers(gdr):
    # a query of NaN sees keys: its row is NaN, in one part or several, and nobody else's
    g, D = gen(31), 64
    for lens, keys in (([5], [90]), ([3], [5000]), ([700], [700])):
        T, TK = sum(lens), sum(keys)
        q, k, v = heads(g, T, 2, 1, D, "dense", TK)[:1] + heads(g, TK, 2, 1, D, "dense", TK)[1:]
        (cu, cuh), (cuk, cukh) = pack(lens), pack(keys)
        clean, cl = gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
        q[1] = NAN
        out, lse = gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
        assert out[1].isnan().all() and lse[:, 1].isnan().all()
        rest = [i for i in range(T) if i != 1]
        assert torch.equal(out[rest], clean[rest]) and torch.equal(lse[:, rest], cl[:, rest])


def test_attention_over_a_long_cache(gdr):
    # keys 2^20 elements apart: their offsets pass 32 bits
    g, n, D = gen(6), 4200, 128
    wide = torch.empty(n, 1 << 20, dtype=BF16, device="cuda")
    k, v = wide[:, :D].unsqueeze(1), wide[:, 1 << 19:(1 << 19) + D].unsqueeze(1)
    k.copy_(randn(g, n, 1, D))
    v.copy_(randn(g, n, 1, D))
    q = randn(g, 3, 4, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack([3]), pack([n])
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
    ro, rl = ref.attention(q.double(), k.double(), v.double(), [3], [n], D ** -0.5, True, 0)
    compare(out, ro, TOL_OUT, "out")
    compare(lse, rl, TOL_LSE, "lse")


def test_attention_refusals(gdr):
    g = gen(2)
    q, k, v = heads(g, 10, 4, 2, 64, "dense", 10)
    cu, cuh = pack([4, 6])
    cuk, cukh = pack([5, 5])
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh)
    dout = torch.zeros_like(out)
    wide = randn(g, 10, 4, 264, dtype=BF16)
    for bad in (lambda: gdr.attn_fwd(q, k[:9], v, cu, cuh), lambda: gdr.attn_fwd(q[:, :3], k, v, cu, cuh), lambda: gdr.attn_fwd(q.float(), k, v, cu, cuh),
                lambda: gdr.attn_fwd(q, k, v, cu, [0, 4, 9]), lambda: gdr.attn_fwd(q, k, v, cu, [0, 11, 10]), lambda: gdr.attn_fwd(q, k, v, cu[:2], cuh),
                lambda: gdr.attn_fwd(q, k, v, cu, cuh, scale=0.0), lambda: gdr.attn_fwd(q, k, v, cu, cuh, scale=NAN),
                lambda: gdr.attn_fwd(q, k, v, cu, cuh, window=-1), lambda: gdr.attn_fwd(q, k, v, cu, cuh, causal=False, window=4),
                lambda: gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk), lambda: gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk[:2], cu_keys_host=[0, 10]),
                lambda: gdr.attn_fwd(q, k[:8], v[:8], cu, cuh, cu_keys=cuk, cu_keys_host=cukh), lambda: gdr.attn_fwd(wide, wide, wide, cu, cuh),
                lambda: gdr.attn_fwd(q.cpu(), k, v, cu, cuh), lambda: gdr.attn_fwd(q.transpose(1, 2), k, v, cu, cuh),
                lambda: gdr.attn_bwd(q, k, v, out, lse.t(), dout, cu, cuh), lambda: gdr.attn_bwd(q, k, v, out, lse, dout[:9], cu, cuh),
                lambda: gdr.attn_bwd(q, k, v, out[:, :2], lse, dout, cu, cuh), lambda: gdr.attn_fwd(q, k, v, cu, cuh, out=out[:5]),
                lambda: gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, grads={"dk": q}), lambda: gdr.attn_fwd(q, k, v, cu, cuh, out=q),
                lambda: gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, grads={"dq": dout}), lambda: gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, grads={"dk": v})):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises((ValueError, RuntimeError)):
        gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, scratch=torch.empty(16, dtype=torch.uint8, device="cuda"))
    e, el = gdr.attn_fwd(q[:0], k[:0], v[:0], cu[:1], [0])
    assert e.shape == (0, 4, 64) and el.shape == (4, 0)
    assert gdr.attn_fwd(q, k, v, cu, cuh, window=1 << 40)[0].equal(out)
    gdr.gdr_check_device()


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
def layer(gdr, x, r, w, b, wqkv, f, cu, cuh, H, HK, D, dout):
    """residual and norm -> q, k, v -> rotary positions -> attention, and the gradients back to x and r."""
    h, y = gdr.lnorm_fwd(x, w, b, residual=r, res_scale=0.5)
    qkv = y @ wqkv
    q, k, v = (qkv[:, a * D:c * D].unflatten(1, (c - a, D)) for a, c in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))
    q, k = gdr.rope_fwd(q, k, f, cu_seqlens=cu)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh)
    gr = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh)
    dq, dk = gdr.rope_bwd(gr["dq"], gr["dk"], f, cu_seqlens=cu)
    dy = torch.cat([t.flatten(1) for t in (dq, dk, gr["dv"])], 1) @ wqkv.t()
    gr = gdr.lnorm_bwd(x, w, b, residual=r, res_scale=0.5, dy=dy)
    return out, gr["dx"], gr["dresidual"], gr["dweight"], gr["dbias"]


def layer_inputs(seed, lens, width, H, HK, D):
    g, T = gen(seed), sum(lens)
    return (randn(g, T, width, dtype=BF16), randn(g, T, width, dtype=BF16), (1 + 0.1 * randn(g, width)).to(BF16), randn(g, width, dtype=BF16),
            (randn(g, width, (H + 2 * HK) * D) * width ** -0.5).to(BF16)), randn(g, T, H, D, dtype=BF16)


def test_the_layer_as_a_whole(gdr):
    lens, width, H, HK, D = [130, 1, 300], 256, 4, 2, 64
    (x, r, w, b, wqkv), dout = layer_inputs(11, lens, width, H, HK, D)
    cu, cuh = pack(lens)
    f = gdr.rope_frequencies(D, scaling="parts", factor=4.0)
    got = layer(gdr, x, r, w, b, wqkv, f, cu, cuh, H, HK, D, dout)
    leaves = [t.double().requires_grad_() for t in (x, r, w, b)]
    _, y = ref.layer_norm(leaves[0], leaves[2], leaves[3], leaves[1], 0.5, 1e-5)
    qkv = y @ wqkv.double()
    q, k, v = (qkv[:, a * D:c * D].unflatten(1, (c - a, D)) for a, c in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))
    pos = torch.cat([torch.arange(n) for n in lens]).cuda()
    q, k = (ref.rotate(t, pos, f, False, 1.0) for t in (q, k))
    ro, _ = ref.attention(q, k, v, lens, lens, D ** -0.5, True, 0)
    want = [ro.detach(), *torch.autograd.grad((ro * dout.double()).sum(), leaves)]
    # y, q/k/v, the turned q and k, out: a bf16 rounding each (2^-8 / sqrt 3 of a binade's lower end, 1.66e-3), which
    # the scores' softmax passes on at about their size (|s| of one); as many again backward
    for t, e, name, tol in zip(got, want, ("out", "dx", "dresidual", "dweight", "dbias"), (8e-3, 1.5e-2, 1.5e-2, 1.5e-2, 1.5e-2)):
        assert rel(t, e) <= tol, (name, rel(t, e))


def test_the_layer_captured_and_on_another_stream(gdr):
    lens, width, H, HK, D = [129, 700], 128, 2, 1, 128
    (x, r, w, b, wqkv), dout = layer_inputs(12, lens, width, H, HK, D)
    cu, cuh = pack(lens)
    f = gdr.rope_frequencies(D)
    args = (x, r, w, b, wqkv, f, cu, cuh, H, HK, D, dout)
    want = layer(gdr, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = layer(gdr, *args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(gdr, *args)
    x.copy_(x.flip(0))
    new = layer(gdr, *args)
    graph.replay()
    torch.cuda.synchronize()
    for a, o, n, c in zip(want, other, new, held):
        assert torch.equal(a, o) and torch.equal(n, c) and not torch.equal(a, c)


# ---------------------------------------------------------------------------
# Attention: the kernels' other paths
# ---------------------------------------------------------------------------
MANY = [
    # many documents (found 32 at a time), many short blocks (taken over), few long ones (in
    # parts), every other key tile of a block with few queries
    ([200, 0, 1, 65] * 40, None, 4, 2, 128, True, 0), ([300] * 50, None, 8, 8, 64, True, 100), ([128] * 200, None, 2, 1, 64, False, 0),
    ([2100], None, 1, 1, 128, True, 0), ([1500], None, 8, 1, 64, True, 0), ([3000], None, 2, 2, 64, True, 700),
    ([129, 1], [2500, 300], 1, 1, 128, True, 0), ([3] * 40, [700 + 13 * i for i in range(40)], 8, 2, 128, True, 0),
    ([1] * 200, [1 + (37 * i) % 700 for i in range(200)], 8, 2, 64, True, 0), ([2] * 90, [300 + i for i in range(90)], 3, 3, 64, True, 100),
    ([1] * 300, [150] * 300, 2, 1, 32, False, 0),
    ([100, 30], [1800, 2300], 4, 4, 80, True, 0), ([1] * 3, [6000, 257, 384], 16, 16, 64, True, 300), ([40], [3000], 6, 3, 128, False, 0),
]


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window", MANY)
def test_attention_of_many_and_of_long_documents(gdr, lq, lk, H, HK, D, causal, window):
    test_attention_forward_and_gradients(gdr, lq, lk, H, HK, D, causal, window, "dense")


@pytest.mark.parametrize("D", [128, 64, 20])
def test_attention_without_queries_or_keys(gdr, D):
    g = gen(D)
    (cu, cuh), (none, noneh) = pack([130, 1]), pack([0, 0])
    x, e = randn(g, 131, 4, D, dtype=BF16), torch.empty(0, 2, D, dtype=BF16, device="cuda")
    out, lse = gdr.attn_fwd(x, e, e, cu, cuh, cu_keys=none, cu_keys_host=noneh)
    assert (out == 0).all() and (lse == -math.inf).all()
    got = gdr.attn_bwd(x, e, e, out, lse, x, cu, cuh, cu_keys=none, cu_keys_host=noneh)
    assert (got["dq"] == 0).all() and got["dk"].shape == e.shape
    k, eq = x[:, :2].contiguous(), torch.empty(0, 4, D, dtype=BF16, device="cuda")
    out, lse = gdr.attn_fwd(eq, k, k, none, noneh, cu_keys=cu, cu_keys_host=cuh)
    got = gdr.attn_bwd(eq, k, k, out, lse, eq, none, noneh, cu_keys=cu, cu_keys_host=cuh)
    assert out.shape == eq.shape and (got["dk"] == 0).all() and (got["dv"] == 0).all()


@pytest.mark.parametrize("H,HK", [(128, 1), (256, 2), (48, 3), (7, 7)])
def test_attention_of_many_heads_a_key_head(gdr, H, HK):
    # one token of each document: up to 128 heads side by side in a tile
    g, keys, D = gen(H), [5, 400, 131], 64
    q, k, v = randn(g, 3, H, D, dtype=BF16), *(randn(g, sum(keys), HK, D, dtype=BF16) for _ in range(2))
    dout = randn(g, 3, H, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack([1, 1, 1]), pack(keys)
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    ro, rl = ref.attention(*leaves, [1, 1, 1], keys, D ** -0.5, True, 0)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
    compare(out, ro.detach(), TOL_OUT, "out")
    compare(lse, rl.detach(), TOL_LSE, "lse")
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
    for n, r in zip(("dq", "dk", "dv"), torch.autograd.grad((ro * dout.double()).sum(), leaves)):
        compare(got[n], r, TOL_GRAD, n)


def test_attention_reads_nothing_of_its_scratch_before_writing_it(gdr):
    g, T, H, HK, D = gen(21), 2600, 2, 1, 128
    q, k, v = heads(g, T, H, HK, D, "dense", T)
    dout = randn(g, T, H, D, dtype=BF16)
    cu, cuh = pack([2590, 10])
    fwd, bwd = gdr.attn_workspace_bytes(T, T, H, HK, D, cuh)
    assert fwd > 0 and bwd > T * H * 4 + 256  # in parts
    dirty = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (fwd, bwd)]  # (NaN in every type)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh)
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh)
    out2, lse2 = gdr.attn_fwd(q, k, v, cu, cuh, scratch=dirty[0])
    got2 = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, scratch=dirty[1])
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and all(torch.equal(got[n], got2[n]) for n in got)


def test_attention_on_two_streams_at_once_and_captured(gdr):
    g, H, HK, D = gen(22), 2, 1, 64
    cases = []
    for lens in ([2300], [300] * 30):  # in parts; blocks that take over others' items
        T = sum(lens)
        cases.append((heads(g, T, H, HK, D, "dense", T), randn(g, T, H, D, dtype=BF16), pack(lens)))

    def run(case):
        (q, k, v), dout, pk = case
        out, lse = gdr.attn_fwd(q, k, v, *pk)
        return out, lse, *gdr.attn_bwd(q, k, v, out, lse, dout, *pk).values()

    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(run(c))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2])), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [run(c) for c in cases]
    for c in cases:
        c[0][0].copy_(c[0][0].flip(0))
    new = [run(c) for c in cases]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, new):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    gdr.gdr_check_device()


def test_attention_leaves_what_lies_around_its_outputs(gdr):
    # outputs as parts of larger tensors: rows before and behind keep their values
    g, lens, H, HK, D = gen(23), [70, 200, 1], 3, 1, 96
    T = sum(lens)
    cu, cuh = pack(lens)
    q, k, v = heads(g, T, H, HK, D, "dense", T)
    dout = randn(g, T, H, D, dtype=BF16)

    def room(n, h):
        t = torch.full((n + 6, h, D), 3.0, dtype=BF16, device="cuda")
        return t, t[3:-3]
    wide_out, out = room(T, H)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, out=out)
    wides, grads = {}, {}
    for n, h in (("dq", H), ("dk", HK), ("dv", HK)):
        wides[n], grads[n] = room(T, h)
    gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, grads=grads)
    plain, _ = gdr.attn_fwd(q, k, v, cu, cuh)
    assert torch.equal(out, plain)
    for t in (wide_out, *wides.values()):
        assert (t[:3] == 3).all() and (t[-3:] == 3).all()


def test_calls_on_a_stream_argument(gdr):
    g, T = gen(24), 300
    q, k, v = heads(g, T, 2, 2, 64, "dense", T)
    cu, cuh = pack([T])
    x, w = randn(g, T, 512, dtype=BF16), randn(g, 512, dtype=BF16)
    f = gdr.rope_frequencies(64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, stream=s)
    grads = gdr.attn_bwd(q, k, v, out, lse, q, cu, cuh, stream=s)
    _, y = gdr.lnorm_fwd(x, w, stream=s)
    dx = gdr.lnorm_bwd(x, w, dy=x, stream=s)["dx"]
    turned, _ = gdr.rope_fwd(q, None, f, cu_seqlens=cu, stream=s)
    back, _ = gdr.rope_bwd(turned, None, f, cu_seqlens=cu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    out2, lse2 = gdr.attn_fwd(q, k, v, cu, cuh)
    assert torch.equal(out, out2) and torch.equal(grads["dk"], gdr.attn_bwd(q, k, v, out2, lse2, q, cu, cuh)["dk"])
    assert torch.equal(y, gdr.lnorm_fwd(x, w)[1]) and torch.equal(dx, gdr.lnorm_bwd(x, w, dy=x)["dx"])
    # there and back: two bf16 roundings
    assert rel(back, q) <= 2 * 2.5e-3


def test_single_tokens_follow_the_prompt(gdr):
    # the last token of each document alone against its keys, and the document's last row
    g, lens, H, HK, D = gen(25), [1, 130, 1000, 257, 64], 8, 2, 128
    T = sum(lens)
    q, k, v = heads(g, T, H, HK, D, "dense", T)
    cu, cuh = pack(lens)
    for window in (0, 100):
        whole, lse = gdr.attn_fwd(q, k, v, cu, cuh, window=window)
        last = torch.tensor(cuh[1:], device="cuda") - 1
        one, ocu = pack([1] * len(lens))
        out, ol = gdr.attn_fwd(q[last], k, v, one, ocu, window=window, cu_keys=cu, cu_keys_host=cuh)
        assert rel(out, whole[last]) <= 2 * TOL_OUT and rel(ol, lse[:, last]) <= TOL_LSE
