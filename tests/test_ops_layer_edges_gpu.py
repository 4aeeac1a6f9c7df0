"""The attention layer's operators on the GPU where they once went wrong: against the plain FP64
references of layer_ref.py, or against themselves."""
import numpy as np
import pytest
import torch

import layer_ref as ref
from test_ops_layer_gpu import ATTN, BF16, F32, MANY, NAN, full, gdr, gen, heads, pack, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 64])
def test_documents_written_by_the_kernel_before(gdr, D):
    # no queries: dk and dv are zero in the rows that cu_keys names, which the kernel before writes
    # as it ends, though kernels behind it may begin early: the integers pass through layer norm's
    # dx = dh (dy = 0) as they are
    g, HK, rows, width = gen(D), 2, 20000, 512
    lens = [700, 0, 129, 300]
    (_, cuh), n = pack(lens), sum(lens)
    none, noneh = pack([0] * len(lens))
    dh = torch.zeros(rows, width, device="cuda")
    dh.view(torch.int32)[-1, :len(cuh)] = torch.tensor(cuh, dtype=torch.int32, device="cuda")
    x, dy = randn(g, rows, width), torch.zeros(rows, width, device="cuda")
    k, q = randn(g, n, HK, D, dtype=BF16), torch.empty(0, 4, D, dtype=BF16, device="cuda")
    lse = torch.empty(4, 0, device="cuda")
    for _ in range(5):
        dx = torch.zeros(rows, width, device="cuda")
        grads = {name: full((n, HK, D), BF16) for name in ("dk", "dv")}
        torch.cuda.synchronize()
        gdr.lnorm_bwd(x, dy=dy, dh=dh, grads={"dx": dx})
        cuk = dx.view(torch.int32)[-1, :len(cuh)]
        got = gdr.attn_bwd(q, k, k, q, lse, q, none, noneh, cu_keys=cuk, cu_keys_host=np.asarray(cuh, dtype=np.int32), grads=grads)
        assert (got["dk"] == 0).all() and (got["dv"] == 0).all()
        assert cuk.tolist() == cuh


@pytest.mark.parametrize("D,H,HK", [(128, 2, 1), (64, 2, 2)])
def test_a_document_does_not_depend_on_its_neighbours(gdr, D, H, HK):
    # a tile reaches into the next document, whose queries must not move anything of this one's, not
    # even a rounding: queries 1000 times as large behind it, whose scores grow along its keys
    g, lens = gen(D + H), [228, 100, 290, 60, 1, 130]
    T = sum(lens)
    cu, cuh = pack(lens)
    q, k, v = heads(g, T, H, HK, D, "dense", T)
    dout = randn(g, T, H, D, dtype=BF16)
    k = (k.float() * torch.linspace(0.5, 2, T, device="cuda")[:, None, None]).to(BF16)
    base = gdr.attn_fwd(q, k, v, cu, cuh)
    grads = gdr.attn_bwd(q, k, v, *base, dout, cu, cuh)
    q2, d2 = q.clone(), dout.clone()
    for n in (1, 3, 5):
        q2[cuh[n]:cuh[n + 1]] *= 1000
        d2[cuh[n]:cuh[n + 1]] *= 1000
    out = gdr.attn_fwd(q2, k, v, cu, cuh)
    got = gdr.attn_bwd(q2, k, v, *out, d2, cu, cuh)
    for n in (0, 2, 4):
        rows = slice(cuh[n], cuh[n + 1])
        assert torch.equal(out[0][rows], base[0][rows]) and torch.equal(out[1][:, rows], base[1][:, rows]), n
        for name in got:
            assert torch.equal(got[name][rows], grads[name][rows]), (n, name)


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_that_are_not_finite(gdr, interleaved):
    # cos and sin of what is no number, or has no end, are no numbers: at every position, 0 among them
    g = gen(7)
    f = torch.tensor([1.0, float("nan"), 0.5, float("inf"), 0.0, -float("inf"), -3.0, 2.0 ** 127], device="cuda")
    pos = torch.tensor([0, 1, -5, 1 << 30], dtype=torch.int32, device="cuda")
    q = randn(g, 4, 3, 18)
    bad = torch.tensor([1, 3, 5], device="cuda")
    cols = torch.cat([2 * bad, 2 * bad + 1] if interleaved else [bad, bad + 8])
    rest = torch.tensor([c for c in range(18) if c not in cols.tolist()], device="cuda")
    sane = torch.where(torch.isfinite(f), f, 0.0)
    for turn in (gdr.rope_fwd, gdr.rope_bwd):
        y, _ = turn(q, None, f, positions=pos, interleaved=interleaved)
        want, _ = turn(q, None, sane, positions=pos, interleaved=interleaved)
        assert y[..., cols].isnan().all()
        assert torch.equal(y[..., rest], want[..., rest])


@pytest.mark.parametrize("f,turns", [(1.0, 2.0 ** -32), (255.0, 2.0 ** -32), (1e4, 2.0 ** -27), (1e6, 2.0 ** -20)])
def test_angles_of_fast_frequencies(gdr, f, turns):
    # the angle modulo a turn against integers of any size: off by 2^-32 turns up to 256 radians a
    # token, by 2^-40 of the frequency beyond; its sine and cosine by FP32's rounding of the fraction
    # (2^-25 turns) and of the values besides
    positions = [1, 12345, 2 ** 30 + 7, 2 ** 31 - 1, -(2 ** 31)]
    digits = 2 ** 200 * 10 ** 60 // (2 * 3141592653589793238462643383279502884197169399375105820974944)  # 2^200 / (2 pi)
    num, den = float(torch.tensor(f, dtype=F32)).as_integer_ratio()
    q = torch.zeros(len(positions), 1, 2, device="cuda")
    q[..., 0] = 1
    y, _ = gdr.rope_fwd(q, None, torch.tensor([f], device="cuda"), positions=torch.tensor(positions, dtype=torch.int32, device="cuda"))
    for p, row in zip(positions, y[:, 0].double().cpu().tolist()):
        fraction = (p * num * digits // den) % 2 ** 200 / 2 ** 200
        off = 2 * np.pi * (turns + 2.0 ** -25) + 2 * 2.0 ** -24
        assert abs(row[0] - np.cos(2 * np.pi * fraction)) <= off and abs(row[1] - np.sin(2 * np.pi * fraction)) <= off, (f, p)


def gradients(q, k, v, dout, lq, lk, scale, causal, window):
    """FP64 gradients from the formulas, and for every row of each the size of its terms (the root of the
    sum of their squares) and of what FP32's products leave of it where dP - delta cancels."""
    G, a, b = q.shape[1] // k.shape[1], 0, 0
    grads, sizes, floors = ([torch.zeros_like(t) for t in (q, k, v)], [torch.zeros(t.shape[:2], dtype=t.dtype, device=t.device) for t in (q, k, v)],
                            [torch.zeros(t.shape[:2], dtype=t.dtype, device=t.device) for t in (q, k, v)])
    for n, m in zip(lq, lk):
        for h in range(q.shape[1]):
            Q, K, V, dO = q[a:a + n, h], k[b:b + m, h // G], v[b:b + m, h // G], dout[a:a + n, h]
            s = scale * Q @ K.T
            if causal:
                gap = torch.arange(n, device=q.device)[:, None] + (m - n) - torch.arange(m, device=q.device)
                s = s.masked_fill((gap < 0) | (gap >= window) if window else gap < 0, -float("inf"))
            p = torch.where((s == -float("inf")).all(-1, keepdim=True), 0.0, torch.softmax(s, -1)) if m else s
            dp = dO @ V.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            # dP and delta are off by 2^-20 of |dout| |v| at most: sums of up to 128 products in FP32
            off = p * (dO.norm(dim=-1)[:, None] * V.norm(dim=-1).max() * 2.0 ** -20) if m else p
            squares = lambda x, y: x.square() @ y.square().sum(-1)  # noqa: E731
            for i, (rows, hh, g, size, floor) in enumerate((
                    (slice(a, a + n), h, scale * ds @ K, scale ** 2 * squares(ds, K), scale ** 2 * squares(off, K)),
                    (slice(b, b + m), h // G, scale * ds.T @ Q, scale ** 2 * squares(ds.T, Q), scale ** 2 * squares(off.T, Q)),
                    (slice(b, b + m), h // G, p.T @ dO, squares(p.T, dO), 0 * squares(p.T, dO)))):
                grads[i][rows, hh] += g
                sizes[i][rows, hh] += size
                floors[i][rows, hh] += floor
        a, b = a + n, b + m
    return grads, [t.sqrt() for t in sizes], [t.sqrt() for t in floors]


PEAKED = [
    # in parts; taken over; few keys a block, gone through twice; keys of one tile; heads side by side; one query a warp
    ([2000], None, 2, 1, 128, True, 0), ([300] * 40, None, 4, 4, 64, True, 0), ([700, 20, 1, 129], None, 4, 2, 128, True, 200),
    ([257, 300], None, 4, 4, 128, False, 0), ([100, 128, 7, 2, 1], None, 2, 2, 128, True, 0), ([1] * 3, [5000, 3, 129], 8, 2, 64, True, 0),
    ([3] * 60, [300 + 7 * i for i in range(60)], 4, 2, 80, True, 0), ([300, 157, 1, 300], None, 4, 4, 64, True, 0),
    ([900], None, 1, 1, 128, False, 0), ([640, 129], None, 8, 8, 128, True, 0), ([400, 140], None, 2, 1, 33, True, 0),
]


@pytest.mark.parametrize("sharp", [1, 4, 8, 32])
@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window", PEAKED)
def test_gradients_of_peaked_probabilities(gdr, lq, lk, H, HK, D, causal, window, sharp):
    # scores `sharp` times those of unit inputs: where one key has nearly all, dP - delta is a small
    # difference.  Every row of a gradient by itself: BF16 leaves each term of it within 2^-8 (P, dS) and
    # the row within 2^-8 (its rounding), and what delta may be off by leaves dq within 2^-8: 3 2^-8 of the terms'
    # size together at worst, if all errors lay one way.  Probabilities and dS below the smallest normal
    # number, 2^-126, are zero: 2^-126 of |dP| |q| scale < 2^12 in each of at most 2^13 terms, below 2^-100
    g, keys = gen(sum(lq) + sharp), lk or lq
    T, TK = sum(lq), sum(keys)
    q, k, v = heads(g, T, H, HK, D, "dense", TK)
    dout = randn(g, T, H, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack(lq), pack(keys) if lk else (None, None)
    args = dict(causal=causal, window=window, cu_keys=cuk, cu_keys_host=cukh, scale=sharp * D ** -0.5)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, **args)
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, **args)
    want, sizes, floors = gradients(q.double(), k.double(), v.double(), dout.double(), lq, keys, float(np.float32(sharp * D ** -0.5)), causal, window)
    for name, r, size, floor in zip(("dq", "dk", "dv"), want, sizes, floors):
        t = got[name].double()
        assert torch.isfinite(t).all(), name
        off = (t - r).norm(dim=-1)
        # of the whole: what layer_ref.py derives for independent roundings
        assert off.norm() <= ref.TOL_GRAD * r.norm() + floor.norm(), f"{name}: {float(off.norm() / r.norm()):.3e}"
        floor = floor + 2.0 ** -100
        worst = (off - floor - 3 * 2 ** -8 * size).argmax()
        assert (off <= 3 * 2 ** -8 * size + floor).all(), (name, int(worst), float(off.flatten()[worst]), float(size.flatten()[worst]), float(floor.flatten()[worst]))
    again = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, **args)
    for name in got:
        assert torch.equal(got[name], again[name]), name


def test_gradients_of_many_tiles_formed_again(gdr):
    # 320000 tiles, every one of peaked scores; the last tokens by themselves, which see 128 keys
    g, T, H, D, window, last = gen(17), 640000, 64, 8, 128, 300
    q, k, v = heads(g, T, H, 1, D, "dense", T)
    dout = randn(g, T, H, D, dtype=BF16)
    cu, cuh = pack([T])
    scale = 24 * D ** -0.5
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, scale=scale, window=window)
    dq = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, scale=scale, window=window)["dq"]
    gdr.gdr_check_device()
    for end in (T, T // 2, window + last):
        a, b = end - last, end - last - window
        want, sizes, floors = gradients(*(t[s:end].double() for t, s in ((q, a), (k, b), (v, b), (dout, a))), [last], [last + window],
                                        float(np.float32(scale)), True, window)
        off = (dq[a:end].double() - want[0]).norm(dim=-1)
        assert off.norm() <= ref.TOL_GRAD * want[0].norm() + floors[0].norm(), end
        assert (off <= 3 * 2 ** -8 * sizes[0] + floors[0] + 2.0 ** -100).all(), end


def rows_of_gradients(gdr, lq, lk, H, HK, D, causal, window, layout="dense", scale=None):
    """Every row of dq, dk and dv by itself against FP64, within BF16's roundings of its own terms."""
    g, keys = gen(sum(lq) + 7 * D), lk or lq
    T, TK = sum(lq), sum(keys)
    q, k, v = heads(g, T, H, HK, D, layout, TK)
    dout = randn(g, T, H, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack(lq), pack(lk) if lk else (None, None)
    args = dict(causal=causal, window=window, cu_keys=cuk, cu_keys_host=cukh)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, **args)
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, **args)
    want, sizes, floors = gradients(q.double(), k.double(), v.double(), dout.double(), lq, keys, float(np.float32(D ** -0.5)), causal, window)
    for name, r, size, floor in zip(("dq", "dk", "dv"), want, sizes, floors):
        off = (got[name].double() - r).norm(dim=-1)
        assert (off <= 3 * 2 ** -8 * size + floor + 2.0 ** -100).all(), (name, float((off - floor - 3 * 2 ** -8 * size).max()))
        # and each document's: what layer_ref.py derives for independent roundings of the terms
        for a, b in zip(*((cuh, cuh[1:]) if name == "dq" else (cukh or cuh, (cukh or cuh)[1:]))):
            assert off[a:b].norm() <= ref.TOL_GRAD * size[a:b].norm() + floor[a:b].norm(), (name, a, b)


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window,layout", ATTN)
def test_every_row_of_the_gradients(gdr, lq, lk, H, HK, D, causal, window, layout):
    rows_of_gradients(gdr, lq, lk, H, HK, D, causal, window, layout)


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window", MANY)
def test_every_row_of_the_gradients_of_many_and_of_long_documents(gdr, lq, lk, H, HK, D, causal, window):
    rows_of_gradients(gdr, lq, lk, H, HK, D, causal, window)


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window", [
    ([700, 129], None, 4, 2, 192, True, 0), ([513], None, 2, 1, 256, True, 100), ([300], [900], 2, 2, 256, True, 0),
    ([1, 3], [1500, 260], 4, 1, 136, True, 0), ([400], None, 3, 3, 250, False, 0)])
def test_wide_heads_of_longer_documents(gdr, lq, lk, H, HK, D, causal, window):
    g, keys = gen(D), lk or lq
    q, k, v = heads(g, sum(lq), H, HK, D, "dense", sum(keys))
    (cu, cuh), (cuk, cukh) = pack(lq), pack(lk) if lk else (None, None)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, causal=causal, window=window, cu_keys=cuk, cu_keys_host=cukh)
    ro, rl = ref.attention(q.double(), k.double(), v.double(), lq, keys, D ** -0.5, causal, window)
    assert (out.double() - ro).norm() <= ref.TOL_OUT * ro.norm() and (lse.double() - rl).norm() <= ref.TOL_LSE * rl.norm()
    rows_of_gradients(gdr, lq, lk, H, HK, D, causal, window)


@pytest.mark.parametrize("D", [128, 33])
def test_documents_of_no_queries_are_room_for_others(gdr, D):
    # a cache that grows in place: between the sequences' keys lie documents without queries, which hold
    # what nobody reads (NaN here); a token appended moves the bounds, not the keys
    g, H, HK, room = gen(D), 4, 2, 400
    used = [300, 1, 257, 128]
    cache = torch.full((2, len(used), room, HK, D), NAN, dtype=BF16, device="cuda")
    for i, n in enumerate(used):
        cache[:, i, :n] = randn(g, 2, n, HK, D, dtype=BF16)
    k, v = cache[0].flatten(0, 1), cache[1].flatten(0, 1)
    q = randn(g, len(used), H, D, dtype=BF16)
    for step in range(2):
        cu, cuh = pack([1, 0] * len(used))
        cuk, cukh = pack([n for u in used for n in (u, room - u)])
        out, lse = gdr.attn_fwd(q, k, v, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
        grads = gdr.attn_bwd(q, k, v, out, lse, q, cu, cuh, cu_keys=cuk, cu_keys_host=cukh)
        pk, pv = (torch.cat([t[i, :n] for i, n in enumerate(used)]) for t in cache)
        ro, rl = ref.attention(q.double(), pk.double(), pv.double(), [1] * len(used), used, D ** -0.5, True, 0)
        assert (out.double() - ro).norm() <= ref.TOL_OUT * ro.norm() and (lse.double() - rl).norm() <= ref.TOL_LSE * rl.norm()
        assert torch.isfinite(grads["dq"].float()).all()
        for i, n in enumerate(used):
            for name in ("dk", "dv"):
                rows = grads[name][i * room:(i + 1) * room]
                assert torch.isfinite(rows.float()).all() and (rows[n:] == 0).all(), (name, i)
        for i in range(len(used)):  # one token more each
            cache[:, i, used[i]] = randn(g, 2, HK, D, dtype=BF16)
            used[i] += 1


@pytest.mark.parametrize("lq,lk,H,HK,D,causal,window", [
    ([1] * 4, [1500, 4000, 22, 3223], 8, 1, 24, True, 0), ([2] * 20, [4000, 3000] * 10, 8, 2, 64, True, 0), ([900], None, 2, 2, 128, True, 0), ([300] * 30, None, 4, 2, 64, True, 0),
    ([99, 135, 290, 106], None, 32, 4, 128, True, 300), ([500], None, 4, 4, 64, False, 0)])
@pytest.mark.parametrize("kpart,vpart", [(16.0, 0.5), (4.0, 4.0), (16.0, 16.0), (16.0, 0.0)])
def test_gradients_of_keys_and_values_that_share_a_part(gdr, lq, lk, H, HK, D, causal, window, kpart, vpart):
    # all keys near one vector, all values near another: the first cancels in dq, since a row of dS sums to
    # zero, but not in what dS is off by together; the second makes delta large beside dP - delta.  Terms' size
    # |dS| |k| includes the shared part: P, dS and dq are rounded (3 2^-8), delta leaves 2^-5.5
    g, keys = gen(D + int(kpart + vpart)), lk or lq
    T, TK = sum(lq), sum(keys)
    q, k, v = heads(g, T, H, HK, D, "dense", TK)
    k, v = ((t.float() + part * randn(g, HK, D)).to(BF16) for t, part in ((k, kpart), (v, vpart)))
    dout = randn(g, T, H, D, dtype=BF16)
    (cu, cuh), (cuk, cukh) = pack(lq), pack(lk) if lk else (None, None)
    args = dict(causal=causal, window=window, cu_keys=cuk, cu_keys_host=cukh)
    out, lse = gdr.attn_fwd(q, k, v, cu, cuh, **args)
    got = gdr.attn_bwd(q, k, v, out, lse, dout, cu, cuh, **args)
    want, sizes, floors = gradients(q.double(), k.double(), v.double(), dout.double(), lq, keys, float(np.float32(D ** -0.5)), causal, window)
    for name, r, size, floor in zip(("dq", "dk", "dv"), want, sizes, floors):
        off = (got[name].double() - r).norm(dim=-1)
        limit = (3 * 2 ** -8 + (2 ** -5.5 if name == "dq" else 0.0)) * size + floor + 2.0 ** -100
        assert (off <= limit).all(), (name, float((off / limit).max()))
