"""The attention layer's operators on the GPU where they once went wrong: against the plain FP64
references of layer_ref.py, or against themselves."""
import numpy as np
import pytest
import torch

from test_ops_layer_gpu import BF16, F32, full, gdr, gen, heads, pack, randn  # noqa: F401

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
