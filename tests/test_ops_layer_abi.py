"""The attention layer's operators without a GPU: every refusal of the C ABI comes before any
CUDA call, workspace sizes and frequencies are host arithmetic, the binding refuses host
tensors."""
import ctypes
import math

import numpy as np
import pytest


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_varlen_gb300 as m
    from gated_delta_rule_varlen_gb300 import build

    build.build()
    m.load()
    return m


def P(n=1):
    return 0x10000 * n  # never dereferenced: every call below is refused on the host, or has nothing to do


def cu(*v):
    a = np.array(v, dtype=np.int32)
    return a, a.ctypes.data


def test_lnorm_refusals(gdr):
    lib, bad = gdr.load(), gdr.GDR_INVALID_ARG

    def fwd(dtype=0, R0=3, R1=1, D=64, x=P(), w=P(), wdt=0, y=P()):
        return lib.lnorm_fwd(dtype, R0, R1, D, x, D, D, None, 0, 0, 1.0, w, None, wdt, 1e-5, None, y, None)
    assert fwd(dtype=3) == bad and fwd(wdt=1) == bad and fwd(D=0) == bad and fwd(D=16385) == bad and fwd(R0=-1) == bad
    assert fwd(R1=0) == bad and fwd(x=None) == bad and fwd(y=None) == bad
    assert fwd(R0=0) == gdr.GDR_OK

    def bwd(dy=P(), dres=None, scratch=P(), nbytes=1 << 40, R0=3):
        return lib.lnorm_bwd(0, R0, 1, 64, P(), 64, 64, None, 0, 0, 1.0, P(), 0, 1e-5, None, 0, 0, dy, 64, 64, P(), dres, P(), None,
                             scratch, nbytes, None)
    assert bwd(dy=None) == bad and bwd(dres=P()) == bad and bwd(scratch=None) == bad and bwd(scratch=P() + 8) == bad
    assert bwd(nbytes=64) == gdr.GDR_WORKSPACE_TOO_SMALL
    assert gdr.lnorm_workspace_bytes(128) >= 2 * 128 * 4
    with pytest.raises(ValueError):
        gdr.lnorm_workspace_bytes(0)


def test_rope_refusals(gdr):
    lib, bad = gdr.load(), gdr.GDR_INVALID_ARG

    def turn(dtype=0, q=P(), HQ=2, qo=P(2), k=None, HK=0, ko=None, T=4, D=64, R=64, f=P(3), pos=P(4), c=None, N=0):
        return lib.rope_turn(dtype, q, 128, 64, HQ, qo, 128, 64, k, 64, 64, HK, ko, 64, 64, T, D, R, f, pos, 0, c, N, 0, 1.0, 0, None)
    for call in (dict(dtype=3), dict(q=None), dict(qo=None), dict(HK=1), dict(HK=1, k=P()), dict(T=-1), dict(T=2**31 - 1), dict(D=0),
                 dict(R=63), dict(R=66), dict(D=16384, R=8194), dict(f=None), dict(pos=None), dict(pos=None, c=P(), N=0), dict(HQ=-1),
                 dict(D=2**20, HQ=2**11, R=2)):
        assert turn(**call) == bad, call
    assert turn(T=0, q=None) == gdr.GDR_OK and turn(HQ=0, q=None) == gdr.GDR_OK


def test_rope_frequencies(gdr):
    import torch
    R, base = 64, 10000.0
    f = base ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    close = lambda a, b: torch.testing.assert_close(a.double(), b, rtol=2**-23, atol=0)  # (one rounding to fp32)  # noqa: E731
    close(gdr.rope_frequencies(R, device="cpu"), f)
    close(gdr.rope_frequencies(R, scaling="linear", factor=4.0, device="cpu"), f / 4)
    grown = gdr.rope_frequencies(R, scaling="base", factor=4.0, device="cpu").double()
    assert grown[0] == 1 and abs(float(grown[-1] / f[-1]) - 0.25) < 1e-6  # the fastest left, the slowest divided
    parts = gdr.rope_frequencies(R, scaling="parts", factor=8.0, context=4096, slow=1.0, fast=32.0, device="cpu").double()
    turns = f * 4096 / (2 * math.pi)
    assert torch.allclose(parts[turns >= 32], f[turns >= 32], rtol=1e-6) and torch.allclose(parts[turns <= 1], f[turns <= 1] / 8, rtol=1e-6)
    mid = (turns > 1) & (turns < 32)
    left = (turns[mid] - 1) / 31
    assert mid.any() and torch.allclose(parts[mid], f[mid] * (left + (1 - left) / 8), rtol=1e-6)
    assert gdr.rope_frequencies(0, device="cpu").shape == (0,) and float(gdr.rope_frequencies(2, scaling="base", factor=3.0, device="cpu")) == 1
    for bad in (dict(R=3), dict(R=-2), dict(R=4, scaling="other"), dict(R=4, base=0.0), dict(R=4, factor=-1.0), dict(R=4, fast=1.0)):
        with pytest.raises(ValueError):
            gdr.rope_frequencies(device="cpu", **bad)


def test_attention_refusals(gdr):
    lib, bad, (k, c), (k2, c2) = gdr.load(), gdr.GDR_INVALID_ARG, cu(0, 5, 11), cu(0, 40, 100)

    def fwd(q=P(), kk=P(), v=P(), d=P(9), host=c, dk=None, hk=None, N=2, T=11, TK=11, H=4, HK=2, D=64, scale=1.0, causal=1, window=0, out=P(2),
            lse=P(3), scratch=None, nbytes=0):
        return lib.attn_fwd(q, H * 64, 64, kk, HK * 64, 64, v, HK * 64, 64, d, host, dk, hk, N, T, TK, H, HK, D, scale, causal, window,
                            out, lse, scratch, nbytes, None)
    for call in (dict(q=None), dict(kk=None), dict(v=None), dict(d=None), dict(out=None), dict(lse=None), dict(H=3), dict(HK=0), dict(H=0),
                 dict(D=0), dict(D=257), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1),
                 dict(causal=0, window=3), dict(out=P()), dict(TK=12), dict(dk=P()), dict(hk=c2, TK=100), dict(N=-1), dict(host=None)):
        assert fwd(**call) == bad, call
    assert fwd(T=12, TK=12) == gdr.GDR_BAD_CU_SEQLENS and fwd(dk=P(), hk=c2, TK=99) == gdr.GDR_BAD_CU_SEQLENS
    kd, cd = cu(0, 7, 5, 11)
    assert fwd(host=cd, N=3) == gdr.GDR_BAD_CU_SEQLENS
    z, cz = cu(0)
    assert fwd(q=None, kk=None, v=None, host=cz, N=0, T=0, TK=0, out=None, lse=None) == gdr.GDR_OK
    # a plan in parts needs its scratch
    kl, cl = cu(0, 1)
    km, cm = cu(0, 65536)
    long = dict(host=cl, N=1, T=1, dk=P(), hk=cm, TK=65536)
    assert fwd(**long) == bad and fwd(scratch=P() + 8, nbytes=1 << 30, **long) == bad
    assert fwd(scratch=P(), nbytes=256, **long) == gdr.GDR_WORKSPACE_TOO_SMALL

    def bwd(out=P(2), lse=P(3), dout=P(4), dq=P(5), dk=P(6), dv=P(7), scratch=P(), nbytes=1 << 30):
        return lib.attn_bwd(P(), 256, 64, P(), 128, 64, P(), 128, 64, out, lse, dout, 256, 64, P(9), c, None, None, 2, 11, 11, 4, 2, 64, 1.0, 1,
                            0, dq, dk, dv, scratch, nbytes, None)
    for call in (dict(out=None), dict(lse=None), dict(dout=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(scratch=None),
                 dict(scratch=P() + 16), dict(dq=P()), dict(dq=P(4)), dict(dk=P(2)), dict(dv=P(6)), dict(dq=P(7))):
        assert bwd(**call) == bad, call
    assert bwd(nbytes=16) == gdr.GDR_WORKSPACE_TOO_SMALL
    kt, ct = cu(0, 2**31 - 1)
    assert fwd(host=ct, N=1, T=2**31 - 1, TK=2**31 - 1, H=1, HK=1) == bad  # (tile ends stay 32 bits)


def test_attention_workspace(gdr):
    # delta alone where the blocks are many or none is long: one float a query and head, to 256 bytes
    n = 4096
    fwd, bwd = gdr.attn_workspace_bytes(16 * n, 16 * n, 16, 16, 128, [n * i for i in range(17)])
    assert fwd == 0 and bwd == 16 * n * 16 * 4
    assert gdr.attn_workspace_bytes(11, 11, 4, 2, 64, [0, 5, 11]) == (0, 256)
    # shapes that go one query a warp take no parts
    assert gdr.attn_workspace_bytes(1, 65536, 8, 8, 33, [0, 1], [0, 65536]) == (0, 256)
    # few long blocks: FP32 shares, out and lse of every query and head a part; dQ, or dK and dV
    fwd, bwd = gdr.attn_workspace_bytes(1, 65536, 32, 8, 128, [0, 1], [0, 65536])
    parts, rest = divmod(fwd, 32 * 129 * 4)
    assert rest == 0 and 8 <= parts <= 32
    fwd, bwd = gdr.attn_workspace_bytes(24576, 24576, 1, 1, 128, [0, 24576])
    parts, rest = divmod(fwd, 24576 * 129 * 4)
    assert rest == 0 and 2 <= parts <= 8 and bwd > 24576 * 4
    fwd, bwd = gdr.attn_workspace_bytes(4096, 4096, 8, 1, 128, [0, 4096])
    shares, rest = divmod(bwd - 4096 * 8 * 4, 2 * 4096 * 128 * 4)
    assert rest == 0 and shares >= 4
    for bad in (lambda: gdr.attn_workspace_bytes(11, 11, 3, 2, 64, [0, 11]), lambda: gdr.attn_workspace_bytes(11, 11, 2, 2, 300, [0, 11]),
                lambda: gdr.attn_workspace_bytes(11, 12, 2, 2, 64, [0, 11]), lambda: gdr.attn_workspace_bytes(11, 11, 2, 2, 64, [0, 11], window=-1)):
        with pytest.raises(ValueError):
            bad()


def test_attention_plan_is_quick(gdr):
    # the plan runs twice a call; it looks at blocks only where they are few
    import time
    k, c = cu(*(40 * i for i in range(20001)))
    n, best = ctypes.c_size_t(0), 1.0
    for _ in range(10):
        start = time.perf_counter()
        assert gdr.load().attn_workspace_bytes(int(k[-1]), int(k[-1]), 16, 16, 128, 20000, c, None, 1, 0, ctypes.byref(n), None) == gdr.GDR_OK
        best = min(best, time.perf_counter() - start)
    assert best < 1e-3, best


def test_binding_refuses_host_tensors(gdr):
    import torch
    x, b, c = torch.zeros(4, 8), torch.zeros(4, 2, 8, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdr.lnorm_fwd(x), lambda: gdr.lnorm_bwd(x, dy=x), lambda: gdr.rope_fwd(b, b, torch.zeros(4), cu_seqlens=c),
                 lambda: gdr.rope_bwd(b, None, torch.zeros(4), cu_seqlens=c), lambda: gdr.attn_fwd(b, b, b, c, [0, 4]),
                 lambda: gdr.attn_bwd(b, b, b, b, x, b, c, [0, 4])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
