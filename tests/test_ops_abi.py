"""The operators around the recurrence without a GPU: every refusal of the C ABI
comes before any CUDA call, workspace sizes are host arithmetic, and the
binding refuses tensors that are not on a CUDA device."""
import ctypes

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


def test_sconv_refusals(gdr):
    lib, (k, c) = gdr.load(), cu(0, 5, 11)

    def fwd(dtype=0, x=P(), ldx=64, w=P(), wdtype=0, cuh=c, N=2, T=11, C=64, W=4, out=P()):
        return lib.sconv_fwd(dtype, x, ldx, w, None, wdtype, P(), cuh, N, T, C, W, 1, None, out, None, None)
    bad = gdr.GDR_INVALID_ARG
    assert fwd(dtype=3) == bad and fwd(wdtype=1) == bad and fwd(W=1) == bad and fwd(W=5) == bad and fwd(C=0) == bad
    assert fwd(x=None) == bad and fwd(w=None) == bad and fwd(out=None) == bad and fwd(ldx=63) == bad
    assert fwd(T=10) == gdr.GDR_BAD_CU_SEQLENS
    k2, c2 = cu(0, 6, 5, 11)
    assert fwd(cuh=c2, N=3) == gdr.GDR_BAD_CU_SEQLENS
    z, cz = cu(0)
    assert lib.sconv_fwd(0, None, 64, P(), None, 0, None, cz, 0, 0, 64, 4, 1, None, None, None, None) == gdr.GDR_OK

    def bwd(scratch=P(), nbytes=1 << 30, dweight=P(), dout=P(), ldo=64):
        return lib.sconv_bwd(0, P(), 64, P(), None, 0, P(), c, 2, 11, 64, 4, 1, None, dout, ldo, None, P(), dweight,
                             None, None, scratch, nbytes, None)
    assert bwd(scratch=None) == bad and bwd(scratch=P() + 16) == bad and bwd(dweight=None) == bad
    assert bwd(dout=None) == bad and bwd(ldo=63) == bad
    assert bwd(nbytes=16) == gdr.GDR_WORKSPACE_TOO_SMALL

    def step(B=3, S=3, slots=None, state=P(), out=P()):
        return lib.sconv_step(0, P(), 64, P(), None, 0, state, slots, B, S, 64, 4, 1, out, None)
    assert step(B=4) == bad and step(S=-1, slots=P()) == bad and step(state=None) == bad and step(out=None) == bad
    assert step(B=0) == gdr.GDR_OK


def test_sconv_refuses_outputs_in_place(gdr):
    lib, bad, c = gdr.load(), gdr.GDR_INVALID_ARG, (ctypes.c_int32 * 2)(0, 9)

    def fwd(x=P(), out=P() + 4096, s0=None, st=None):
        return lib.sconv_fwd(0, x, 64, P(), None, 0, P(), c, 1, 9, 64, 4, 1, s0, out, st, None)
    assert fwd(out=P()) == bad and fwd(s0=P(), st=P()) == bad

    def bwd(x=P(), dout=P() + 4096, dx=P() + 8192, s0=None, dst=None, ds0=None):
        return lib.sconv_bwd(0, x, 64, P(), None, 0, P(), c, 1, 9, 64, 4, 1, s0, dout, 64, dst, dx, P(), None, ds0, P(),
                             1 << 40, None)
    assert bwd(dx=P()) == bad and bwd(dx=P() + 4096) == bad and bwd(dst=P(), ds0=P()) == bad and bwd(s0=P(), ds0=P()) == bad


def test_ssm_refusals(gdr):
    lib, (k, c) = gdr.load(), cu(0, 5, 11)
    bad = gdr.GDR_INVALID_ARG

    def fwd(x=P(), ldx=128, dtt=2, ldb=128, cuh=c, N=2, T=11, H=2, Pd=64, G=1, NS=128, out=P(), scratch=P(),
            nbytes=1 << 40):
        return lib.ssm_fwd(x, ldx, P(), dtt, H, P(), P(), ldb, P(), ldb, None, None, 1, P(), cuh, N, T, H, Pd, G, NS,
                           None, out, None, scratch, nbytes, None)
    assert fwd(H=3, G=2) == bad and fwd(Pd=0) == bad and fwd(Pd=257) == bad and fwd(NS=0) == bad and fwd(NS=257) == bad
    assert fwd(dtt=1) == bad and fwd(x=None) == bad and fwd(out=None) == bad and fwd(ldx=127) == bad and fwd(ldb=127) == bad
    assert fwd(T=12) == gdr.GDR_BAD_CU_SEQLENS
    assert fwd(scratch=None) == bad and fwd(scratch=P() + 16) == bad
    assert fwd(nbytes=1024) == gdr.GDR_WORKSPACE_TOO_SMALL

    def step(B=3, S=3, slots=None, state=P()):
        return lib.ssm_step(P(), 128, P(), 2, 2, P(), P(), 128, P(), 128, None, None, 1, state, slots, B, S, 2, 64, 1, 128,
                            P(), None)
    assert step(B=4) == bad and step(state=None) == bad and step(S=-1, slots=P()) == bad
    assert step(B=0) == gdr.GDR_OK


def test_delta_step_refusals(gdr):
    lib, bad = gdr.load(), gdr.GDR_INVALID_ARG

    def step(q=P(), state=P(), slots=None, B=2, S=2, Hqk=2, HV=4, out=P()):
        return lib.gdn_step(q, P(), P(), P(), P(), state, slots, B, S, Hqk, HV, 1.0, 0, out, None)
    assert step(HV=5) == bad and step(Hqk=0) == bad and step(q=None) == bad and step(out=None) == bad
    assert step(state=None) == bad and step(state=P() + 4) == bad and step(B=3) == bad and step(B=-1) == bad
    assert step(B=0) == gdr.GDR_OK
    assert lib.kda_step(None, P(), P(), P(), P(), P(), None, 1, 1, 1, 1.0, 0, P(), None) == bad


def test_norm_refusals(gdr):
    lib, bad = gdr.load(), gdr.GDR_INVALID_ARG

    def fwd(dtype=0, R0=3, D=64, x=P(), act=0, res=None, post=P(), w=None, wdt=0, h=P(), y=None):
        return lib.norm_fwd(dtype, R0, 1, D, x, D, D, None, 0, 0, act, res, D, D, 1.0, post, w, wdt, 1e-6, h, y, None)
    assert fwd(dtype=4) == bad and fwd(wdt=1) == bad and fwd(D=0) == bad and fwd(D=16385) == bad and fwd(act=2) == bad
    assert fwd(x=None) == bad and fwd(post=None) == bad and fwd(h=None) == bad and fwd(y=P()) == bad and fwd(R0=-1) == bad
    assert fwd(R0=0) == gdr.GDR_OK

    def bwd(post=P(), w=None, gate=None, dh=P(), dy=None, dgate=None, dres=None, dw=None, scratch=P(), nbytes=1 << 40):
        return lib.norm_bwd(0, 3, 1, 64, P(), 64, 64, gate, 64, 64, 0, None, 0, 0, 1.0, post, w, 0, 1e-6, dh, 64, 64, dy,
                            64, 64, P(), dgate, dres, dw, None, scratch, nbytes, None)
    assert bwd(dh=None) == bad and bwd(dy=P()) == bad and bwd(dgate=P()) == bad and bwd(dres=P()) == bad
    assert bwd(dw=P()) == bad and bwd(scratch=None) == bad and bwd(scratch=P() + 8) == bad
    assert bwd(nbytes=64) == gdr.GDR_WORKSPACE_TOO_SMALL


def test_sizes_at_the_end_of_32_bits(gdr):
    # tile ends, channels and a token's elements are ints in the kernels: what would pass them is refused
    lib, bad, most = gdr.load(), gdr.GDR_INVALID_ARG, 2**31 - 2**16
    n = ctypes.c_size_t(0)
    for T in (most + 1, 2**31 - 1):
        k, c = cu(0, T)
        assert lib.sconv_fwd(0, P(), 1, P(), None, 0, P(), c, 1, T, 1, 4, 1, None, P(2), None, None) == bad
        assert lib.sconv_bwd(0, P(), 1, P(), None, 0, P(), c, 1, T, 1, 4, 1, None, P(2), 1, None, P(3), P(), None, None, P(),
                             1 << 50, None) == bad
        assert lib.sconv_step(0, P(), 1, P(), None, 0, P(), None, T, T, 1, 4, 1, P(2), None) == bad
        assert lib.sconv_workspace_bytes(T, 1, 4, ctypes.byref(n)) == bad
        assert lib.sconv_workspace_bytes(1, T, 4, ctypes.byref(n)) == bad
        assert lib.ssm_workspace_bytes(T, 1, 1, 1, 1, 1, c, ctypes.byref(n)) == bad
        assert lib.ssm_fwd(P(), 1, P(), 2, 1, P(), P(), 1, P(), 1, None, None, 1, P(), c, 1, T, 1, 1, 1, 1, None, P(2), None,
                           P(), 1 << 50, None) == bad
    k, c = cu(0, 4)
    C = 2**31 - 500
    assert lib.sconv_fwd(0, P(), C, P(), None, 0, P(), c, 1, 4, C, 4, 1, None, P(2), None, None) == bad
    assert lib.sconv_step(0, P(), C, P(), None, 0, P(), None, 1, 1, C, 4, 1, P(2), None) == bad
    H = 2**23  # of 256 columns
    assert lib.ssm_step(P(), 2**31, P(), 2, H, P(), P(), 1, P(), 1, None, None, 1, P(), None, 1, 1, H, 256, 1, 1, P(2), None) == bad
    assert lib.ssm_step(P(), H, P(), 2, H, P(), P(), 2**31, P(), 2**31, None, None, 1, P(), None, 1, 1, H, 1, H, 256, P(2),
                        None) == bad


def test_workspace_sizes(gdr):
    # partial rows of W + 1 sums a channel and tile; tiles of 256 tokens at most, 16 at least
    for T, C, W in ((0, 8, 2), (1, 37, 4), (1000, 64, 3), (32768, 10240, 4)):
        n = gdr.sconv_workspace_bytes(T, C, W)
        tiles = n // ((W + 1) * C * 4)
        assert n == tiles * (W + 1) * C * 4 and tiles >= max(1, T / 320) and tiles <= max(1, -(-T // 16))
    assert gdr.norm_workspace_bytes(128) >= 2 * 128 * 4
    with pytest.raises(ValueError):
        gdr.norm_workspace_bytes(16385)
    with pytest.raises(ValueError):
        gdr.sconv_workspace_bytes(10, 8, 5)
    # the gates of every chunk (an empty document counts as one), 352 floats a chunk and head
    assert gdr.ssm_workspace_bytes(129, 4, 64, 1, 128, [0, 1, 1, 129]) == 3 * 4 * 352 * 4
    # states of segments are added where a document is split over the SMs; few heads, one long document
    whole = 2048 * 4 * 352 * 4
    split = gdr.ssm_workspace_bytes(262144, 4, 64, 1, 128, [0, 262144])
    assert split > whole + 8 * 4 * 64 * 128 * 4
    # sizes that the chunked kernels do not take go token by token, without scratch
    for H, Pd, N in ((4, 33, 128), (4, 64, 130), (4, 64, 256)):
        assert gdr.ssm_workspace_bytes(100, H, Pd, 1, N, [0, 100]) == 0
    with pytest.raises(ValueError):
        gdr.ssm_workspace_bytes(100, 4, 64, 3, 128, [0, 100])
    with pytest.raises(ValueError):
        gdr.ssm_workspace_bytes(100, 4, 64, 1, 128, [0, 99])


def test_scan_scratch_holds_states_of_split_documents_only(gdr):
    # 128k tokens in segments and 1000 documents of 64 tokens, whose states are carried in registers
    H, state = 8, 8 * 64 * 128 * 4
    cu_host = [0] + [131072 + 64 * i for i in range(1001)]
    gates = (1024 + 1000) * H * 352 * 4
    n = gdr.ssm_workspace_bytes(cu_host[-1], H, 64, 1, 128, cu_host)
    assert gates + 2 * state < n < gates + 256 * (state + 4 * H) + 1024  # (at most 256 segments a document)


def test_scan_plan_is_quick_with_many_documents(gdr):
    # the plan runs twice a call: one long document among 4095 of 16 tokens took it 3.8 ms when it went through
    # all documents for every segment length, and takes some 15 us
    import time
    k, c = cu(0, *(131072 + 16 * i for i in range(4096)))
    n, best = ctypes.c_size_t(0), 1.0
    for _ in range(20):
        start = time.perf_counter()
        rc = gdr.load().ssm_workspace_bytes(int(k[-1]), 64, 64, 8, 128, 4096, c, ctypes.byref(n))
        best = min(best, time.perf_counter() - start)
    assert rc == gdr.GDR_OK and best < 5e-4, best


def test_binding_refuses_host_tensors(gdr):
    import torch
    x = torch.zeros(4, 8)
    w = torch.zeros(8, 4)
    c = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdr.sconv_fwd(x, w, None, c, [0, 4]), lambda: gdr.sconv_step(x, w, None, torch.zeros(4, 3, 8)),
                 lambda: gdr.norm_fwd(x, weight=w[:, 0]), lambda: gdr.norm_bwd(x, weight=w[:, 0], dy=x),
                 lambda: gdr.ssm_step(x[:, None].bfloat16(), x, x, x, x, x),
                 lambda: gdr.gdn_step(x[:, None], x, x, x, x, x, 1.0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_exports_are_reachable_from_the_package(gdr):
    from gated_delta_rule_varlen_gb300 import ops
    for name in ops.__all__:
        assert getattr(gdr, name) is getattr(ops, name)
    with pytest.raises(AttributeError):
        gdr.no_such_operator
    assert ctypes.sizeof(ctypes.c_size_t) == 8
