"""The operators around the recurrence (short convolution, selective scan,
single-token forms, norms) on the GPU, against the plain FP64 references of
ops_ref.py: every type, odd sizes and strides, ragged and empty documents,
carried states, inactive rows, gradients by the formulas and by differences,
and the refusals of the binding."""
import pytest
import torch

import ops_ref as ref
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


def rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def full(shape, dtype):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


def strided(t, pad, odd=False):
    """The same values as a slice of wider rows (odd: on no 16-byte boundary)."""
    wide = torch.full((t.shape[0], t[0].numel() + pad + (1 if odd else 0)), 7.0, dtype=t.dtype, device=t.device)
    view = wide[:, (1 if odd else 0):][:, :t[0].numel()]
    view.copy_(t.reshape(t.shape[0], -1))
    return view.unflatten(1, t.shape[1:]) if t.dim() > 2 else view


def pack(lengths):
    cu = cu_of(lengths)
    return torch.tensor(cu, dtype=torch.int32, device="cuda"), cu


# ---------------------------------------------------------------------------
# Short convolution
# ---------------------------------------------------------------------------
RAGGED = [0, 1, 2, 3, 0, 0, 7, 40, 17, 255, 5, 0]
CONV = [
    # lengths, C, W, dtype, bias, silu, states, row padding, odd start, fp32 weights
    (RAGGED, 128, 4, BF16, True, True, True, 0, False, False),
    (RAGGED, 40, 3, F32, True, True, True, 8, False, False),
    (RAGGED, 37, 4, BF16, False, True, True, 3, True, False),
    (RAGGED, 64, 2, F16, True, False, True, 0, False, True),
    ([1], 8, 4, BF16, False, True, False, 0, False, False),
    ([0, 0], 16, 4, BF16, True, True, True, 0, False, False),
    ([2048, 1, 511], 1536, 4, BF16, True, True, False, 64, False, True),
    ([300] * 7, 1025, 3, F32, False, True, True, 0, False, False),
    ([1] * 50, 24, 4, F16, True, True, True, 0, False, False),
    ([1000], 8, 2, BF16, False, False, False, 0, False, False),
]


# channels in pairs: counts and strides of no whole 8 or 16 bytes
CONV += [([1, 33, 0, 7, 300], 1022, 4, BF16, True, True, True, 0, False, False), ([70, 5], 6, 3, F16, False, True, True, 2, False, True),
         ([9, 140], 64, 2, BF16, True, False, True, 2, False, False), ([128, 64], 258, 4, F16, True, True, False, 0, False, False)]


@pytest.mark.parametrize("lengths,C,W,dtype,bias,silu,states,pad,odd,wf32", CONV)
def test_sconv_forward_and_gradients(gdr, lengths, C, W, dtype, bias, silu, states, pad, odd, wf32):
    g, T, n, K = gen(C + W), sum(lengths), len(lengths), W - 1
    x = randn(g, T, C, dtype=dtype)
    wt = F32 if wf32 else dtype
    w = randn(g, C, W).mul(0.5).to(wt)
    b = randn(g, C, dtype=wt) if bias else None
    s0, dst = (randn(g, n, K, C, dtype=dtype) if states else None for _ in range(2))
    dout = randn(g, T, C, dtype=dtype)
    cu, cuh = pack(lengths)
    xs, ds = (strided(t, pad, odd) if (pad or odd) and T else t for t in (x, dout))
    out, st = gdr.sconv_fwd(xs, w, b, cu, cuh, s0=s0, silu=silu, out=full((T, C), dtype), st=full((n, K, C), dtype))
    leaves = [t.double().requires_grad_() if t is not None else None for t in (x, w, b, s0)]
    ro, rs = ref.conv(*leaves[:3], lengths, leaves[3], silu)
    check(out, ro, "out")
    assert torch.equal(st, rs.to(dtype)), "end states are copies"
    grads = {"dx": full((T, C), dtype), "dweight": full((C, W), F32)}
    if bias:
        grads["dbias"] = full((C,), F32)
    if states:
        grads["ds0"] = full((n, K, C), dtype)
    got = gdr.sconv_bwd(xs, w, b, cu, cuh, ds, s0=s0, dst=dst, want_ds0=states, silu=silu, grads=grads)
    total = (ro * dout.double()).sum() + (rs * dst.double()).sum() if states else (ro * dout.double()).sum()
    want = [t for t in leaves if t is not None]
    rg = dict(zip([m for m, t in zip(("dx", "dweight", "dbias", "ds0"), leaves) if t is not None],
                  torch.autograd.grad(total, want, allow_unused=True)))
    for name, r in rg.items():
        check(got[name], torch.zeros_like(got[name]) if r is None else r, name)
    # the same call again gives the same bits
    again = gdr.sconv_bwd(xs, w, b, cu, cuh, ds, s0=s0, dst=dst, want_ds0=states, silu=silu)
    for name in rg:
        assert torch.equal(got[name], again[name]), name


def test_sconv_gradients_by_differences(gdr):
    g, lengths, C, W = gen(1), [5, 0, 33, 2], 24, 4
    T, n = sum(lengths), len(lengths)
    cu, cuh = pack(lengths)
    args = {"x": randn(g, T, C), "w": randn(g, C, W), "b": randn(g, C), "s0": randn(g, n, W - 1, C)}
    dout, dst = randn(g, T, C), randn(g, n, W - 1, C)

    def loss(a):
        out, st = gdr.sconv_fwd(a["x"], a["w"], a["b"], cu, cuh, s0=a["s0"])
        return float((out.double() * dout.double()).sum() + (st.double() * dst.double()).sum())

    got = gdr.sconv_bwd(args["x"], args["w"], args["b"], cu, cuh, dout, s0=args["s0"], dst=dst, want_ds0=True)
    for name, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("s0", "ds0")):
        v = randn(g, *args[name].shape)
        eps = 1e-2
        up, down = ({**args, name: args[name] + s * eps * v} for s in (1, -1))
        diff = (loss(up) - loss(down)) / (2 * eps)
        inner = float((got[grad].double() * v.double()).sum())
        # truncation eps^2 / 6 of a third derivative below 1, FP32 rounding 1e-7 sum / eps
        assert abs(diff - inner) <= 2e-3 * float(got[grad].double().norm() * v.double().norm()) + 1e-2, (name, diff, inner)


@pytest.mark.parametrize("B,C,W,dtype,bias,silu,pad,odd", [
    (1, 1536, 4, BF16, False, True, 0, False), (5, 37, 3, F32, True, True, 2, True), (64, 128, 2, F16, True, False, 0, False),
    (3, 1, 4, BF16, True, True, 0, False), (300, 16, 4, BF16, False, True, 16, False)])
def test_sconv_step_follows_the_prompt(gdr, B, C, W, dtype, bias, silu, pad, odd):
    g, S = gen(B + C), B + 4
    w, b = randn(g, C, W, dtype=dtype), randn(g, C, dtype=dtype) if bias else None
    state = randn(g, S, W - 1, C, dtype=dtype)
    slots = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, S  # inactive rows
    before, live = state.clone(), (slots >= 0) & (slots < S)
    r = before.double()[torch.where(live, slots, 0).long()]
    for step in range(W + 1):  # until the start states have left the window
        x = randn(g, B, C, dtype=dtype)
        out = gdr.sconv_step(strided(x, pad, odd) if pad else x, w, b, state, slots=slots, silu=silu, out=full((B, C), dtype))
        xx = torch.cat([r, x.double()[:, None]], 1)
        z = (xx * w.double().t()).sum(1) + (b.double() if bias else 0)
        check(out, torch.where(live[:, None], z * torch.sigmoid(z) if silu else z, torch.zeros_like(z)), f"step {step}")
        r = xx[:, 1:]
    used = slots[live].long()
    assert torch.equal(state[used], r[live].to(dtype))
    rest = torch.ones(S, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(state[rest], before[rest]), "a state of no row was touched"


def test_silu_and_sigmoid_keep_their_bits(gdr):
    # FP32, element by element over the whole range: the exponential (2 ulp), the factor of its argument's rounding
    # and its product with it, 1 + y and z s (half an ulp each) and the reciprocal (1 ulp) add up to 5 ulp of 2^-23
    z = torch.cat([torch.linspace(-86, 86, 4001), torch.linspace(-1, 1, 1003)]).cuda()
    n, zd, W = z.numel(), z.double(), 3
    w = torch.zeros(n, W, device="cuda")
    w[:, W - 1] = 1
    s = torch.exp(-torch.nn.functional.softplus(-zd, threshold=1e9))

    def off(got, want):
        assert torch.isfinite(got).all()
        return float(((got.double() - want).abs() / want.abs().clamp_min(1e-300)).max())
    most = 5 * 2.0 ** -23
    assert off(gdr.sconv_step(z[None], w, None, torch.zeros(1, W - 1, n, device="cuda"))[0], zd * s) <= most
    cu = pack([2])
    assert off(gdr.sconv_fwd(torch.stack([z, z]), w, None, *cu)[0][1], zd * s) <= most
    one, zero = torch.ones_like(z), torch.zeros_like(z)
    for act, want in (("silu", zd * s), ("sigmoid", s)):
        h, _ = gdr.norm_fwd(one[None], gate=z[None], act=act, residual=zero[None])
        assert off(h[0], want) <= most, act
    inf = torch.tensor([float("inf"), -float("inf"), NAN], device="cuda")
    h, _ = gdr.norm_fwd(torch.ones(1, 3, device="cuda"), gate=inf[None], act="sigmoid", residual=torch.zeros(1, 3, device="cuda"))
    assert h[0, 0] == 1 and h[0, 1] == 0 and torch.isnan(h[0, 2])


def test_sconv_infinities_stay_in_their_document(gdr):
    # an inf or NaN before a document's start, or in its neighbour channel, reaches no other output
    g, C, lengths = gen(3), 16, [4, 4, 4]
    x = randn(g, 12, C)
    cu, cuh = pack(lengths)
    w = randn(g, C, 2)
    base, _ = gdr.sconv_fwd(x, w, None, cu, cuh)
    bad = x.clone()
    bad[3] = float("inf")
    bad[8, 5] = NAN
    out, _ = gdr.sconv_fwd(bad, w, None, cu, cuh)
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[3], keep[8:10, 5] = False, False
    assert torch.equal(out[keep], base[keep])


# ---------------------------------------------------------------------------
# Selective scan
# ---------------------------------------------------------------------------
def scan_inputs(g, T, H, P, G, N, dt_dtype, pad=0, odd=False):
    def rows(*shape):
        t = torch.nn.functional.silu(randn(g, *shape)).to(BF16)
        return strided(t, pad, odd) if pad and shape[0] else t
    x, B, C = rows(T, H, P), rows(T, G, N), rows(T, G, N)
    dt = randn(g, T, H, dtype=dt_dtype)
    A = -(0.5 + 8 * rand(g, H))
    D = randn(g, H)
    bias = -4 + 3 * rand(g, H)
    return x, dt, A, B, C, D, bias


SCAN = [
    # lengths, H, P, G, N, dt dtype, skip, states, row padding, odd start
    ([1, 63, 64, 0, 65, 129, 300], 4, 64, 1, 128, F32, True, True, 0, False),
    ([130, 1, 0, 257], 6, 64, 2, 128, BF16, True, False, 16, False),
    ([200], 2, 128, 2, 64, BF16, False, True, 0, False),
    ([0, 0], 2, 64, 1, 128, F32, True, True, 0, False),
    ([70, 2], 3, 40, 1, 24, F32, True, True, 0, False),
    ([97, 33], 2, 33, 1, 17, BF16, True, True, 5, True),
    ([150], 2, 256, 1, 256, F32, True, True, 0, False),
    ([1] * 9, 8, 32, 4, 16, BF16, True, True, 0, False),
    ([700, 13], 8, 64, 8, 64, F32, True, True, 64, False),
    ([260, 5], 2, 80, 1, 96, F32, True, True, 0, False),
    ([100], 1, 1, 1, 1, F32, False, False, 0, False),
]


@pytest.mark.parametrize("lengths,H,P,G,N,dt_dtype,skip,states,pad,odd", SCAN)
def test_ssm_prompt(gdr, lengths, H, P, G, N, dt_dtype, skip, states, pad, odd):
    g, T, n = gen(H * P + N), sum(lengths), len(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, T, H, P, G, N, dt_dtype, pad, odd)
    D = D if skip else None
    h0 = randn(g, n, H, N, P) if states else None
    cu, cuh = pack(lengths)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, D=D, dt_bias=bias, h0=h0, out=full((T, H, P), BF16),
                          ht=full((n, H, N, P), F32))
    torch.cuda.synchronize()
    gdr.gdr_check_device()
    act = torch.nn.functional.softplus(dt.double() + bias.double(), threshold=100.0)
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), None if D is None else D.double(), lengths,
                      None if h0 is None else h0.double())
    if T:
        check(out, ro, "out")
    check(ht, rh, "ht")
    again, ht2 = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, D=D, dt_bias=bias, h0=h0)
    assert torch.equal(out, again) and torch.equal(ht, ht2), "the same call again gives the same bits"


@pytest.mark.parametrize("lengths,H,G", [([4096], 2, 1), ([1500, 2500, 3], 4, 2)])
def test_ssm_prompt_equals_its_pieces(gdr, lengths, H, G):
    # a long prompt, and the same prompt handed over in two calls with the state carried
    g, P, N, T = gen(5), 64, 128, sum(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, T, H, P, G, N, F32)
    cu, cuh = pack(lengths)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, D=D, dt_bias=bias)
    act = torch.nn.functional.softplus(dt.double() + bias.double())
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), D.double(), lengths, None)
    check(out, ro, "out")
    check(ht, rh, "ht")
    at = 0
    for i, m in enumerate(lengths):
        cut = min(m, 777)
        one, two = pack([cut]), pack([m - cut])
        part = [t[at:at + cut] for t in (x, dt, B, C)]
        o1, s1 = gdr.ssm_fwd(part[0], part[1], A, part[2], part[3], *one, D=D, dt_bias=bias)
        part = [t[at + cut:at + m] for t in (x, dt, B, C)]
        o2, s2 = gdr.ssm_fwd(part[0], part[1], A, part[2], part[3], *two, D=D, dt_bias=bias, h0=s1)
        check(torch.cat([o1, o2]), ro[at:at + m], "pieces")
        check(s2[0], rh[i], "carried state")
        at += m


@pytest.mark.parametrize("lengths,H,P,G,N", [
    ([3000], 3, 64, 1, 96),        # an odd number of heads a group
    ([40, 2900], 3, 128, 3, 64),   # one head a group, in two column blocks
    ([2700], 2, 80, 2, 24),        # the second column block part empty, one block of state rows
    ([2600, 1], 5, 72, 1, 128),
])
def test_ssm_prompt_in_segments(gdr, lengths, H, P, G, N):
    g, T, n = gen(H * P + N + 1), sum(lengths), len(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, T, H, P, G, N, F32)
    h0, cu, cuh = randn(g, n, H, N, P), *pack(lengths)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, D=D, dt_bias=bias, h0=h0, ht=full((n, H, N, P), F32))
    torch.cuda.synchronize()
    gdr.gdr_check_device()
    act = torch.nn.functional.softplus(dt.double() + bias.double())
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), D.double(), lengths, h0.double())
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("lengths,H,P,G,N,odd", [
    ([32, 1, 0, 31, 4], 4, 64, 2, 128, False),    # every document short
    ([33, 1, 0, 31, 4], 4, 64, 2, 128, False),    # one a token longer
    ([2, 5], 2, 72, 1, 40, False),
    ([7, 32, 3], 3, 66, 1, 33, False),
    ([30, 9], 2, 44, 1, 200, True),
])
def test_ssm_prompt_short(gdr, lengths, H, P, G, N, odd):
    g, T, n = gen(H + P * N), sum(lengths), len(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, T, H, P, G, N, F32, 0, odd)
    h0, cu, cuh = randn(g, n, H, N, P), *pack(lengths)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, D=D, dt_bias=bias, h0=h0, out=full((T, H, P), BF16),
                          ht=full((n, H, N, P), F32))
    torch.cuda.synchronize()
    gdr.gdr_check_device()
    act = torch.nn.functional.softplus(dt.double() + bias.double())
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), D.double(), lengths, h0.double())
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("lengths", [[3000], [200, 0, 129, 40], [20, 3, 0]])
def test_ssm_prompt_states_in_place(gdr, lengths):
    g, P, N, H, n = gen(12), 64, 128, 2, len(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, sum(lengths), H, P, 1, N, F32)
    h0, cu = randn(g, n, H, N, P), pack(lengths)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *cu, D=D, dt_bias=bias, h0=h0)
    pool = h0.clone()
    out2, ht2 = gdr.ssm_fwd(x, dt, A, B, C, *cu, D=D, dt_bias=bias, h0=pool, ht=pool)
    assert ht2 is pool and torch.equal(out, out2) and torch.equal(ht, pool)


@pytest.mark.parametrize("lengths,H,P,G,N,states", [
    ([9000, 2500, 70], 3, 64, 1, 128, True), ([20000], 8, 64, 2, 64, True), ([5000, 0, 4999], 2, 80, 1, 96, True),
    ([7000, 33], 4, 64, 1, 128, False), ([40, 9000, 0, 200, 5000, 33, 1, 6000, 129], 2, 64, 1, 64, True),
    ([5] * 40 + [6000] + [130, 0] * 35 + [5000, 7], 1, 64, 1, 64, True)])
def test_ssm_prompt_in_segments_in_place(gdr, lengths, H, P, G, N, states):
    # a split document's first segment takes its start state from the merge, whatever its last segment has
    # written over h0 by then: in place, out of place and without h0 but zeros, the same bits
    g, n = gen(34), len(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, sum(lengths), H, P, G, N, F32)
    h0, cu = 20 * randn(g, n, H, N, P) if states else torch.zeros(n, H, N, P, device="cuda"), pack(lengths)
    assert gdr.ssm_workspace_bytes(sum(lengths), H, P, G, N, cu[1]) > 4 * 352 * H * sum(max(1, -(-m // 128)) for m in lengths) + 1024
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *cu, D=D, dt_bias=bias, h0=h0 if states else None)
    for _ in range(5):
        pool = h0.clone()
        out2, ht2 = gdr.ssm_fwd(x, dt, A, B, C, *cu, D=D, dt_bias=bias, h0=pool, ht=pool)
        assert ht2 is pool and torch.equal(out, out2) and torch.equal(ht, pool)
    act = torch.nn.functional.softplus(dt.double() + bias.double())
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), D.double(), lengths, h0.double())
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("D", [128, 1021, 2048, 5120, 9000])
def test_norm_in_place(gdr, D):
    g = gen(D)
    x, r = randn(g, 50, D, dtype=BF16), randn(g, 50, D, dtype=BF16)
    w = (1 + 0.2 * randn(g, D)).to(BF16)
    h, y = gdr.norm_fwd(x, weight=w, post_weight=w, residual=r)
    x2, r2 = x.clone(), r.clone()
    gdr.norm_fwd(x2, weight=w, post_weight=w, residual=r2, h=r2, y=x2)
    assert torch.equal(h, r2) and torch.equal(y, x2)


def test_ssm_prompt_carries_nan(gdr):
    # a NaN reaches every later token of its own document and head, across segments, and no other
    g, P, N, H, lengths = gen(8), 64, 128, 2, [200, 3000]
    x, dt, A, B, C, D, bias = scan_inputs(g, sum(lengths), H, P, 1, N, F32)
    at = 200 + 131
    x[at, 1, 7] = float("nan")
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *pack(lengths), D=D, dt_bias=bias)
    assert torch.isnan(out[at:, 1, 7]).all() and torch.isnan(ht[1, 1, :, 7]).all()
    assert torch.isfinite(out[:, 0]).all() and torch.isfinite(out[:200]).all() and torch.isfinite(ht[0]).all()
    assert torch.isfinite(out[200:at // 128 * 128]).all()  # earlier tokens of the same chunk may see it


@pytest.mark.parametrize("decay,dtv", [(0.0, 0.05), (-1e4, 1.0), (-16.0, 20.0), (-1e-3, 1e-3)])
def test_ssm_prompt_extreme_decays(gdr, decay, dtv):
    # no decay at all, states that vanish within a token, and both ends between, without softplus
    g, lengths, H, P, N = gen(6), [130, 64], 2, 64, 128
    T = sum(lengths)
    x, dt, A, B, C, D, bias = scan_inputs(g, T, H, P, 1, N, F32)
    dt = dtv * (0.5 + rand(g, T, H))
    A = torch.full_like(A, decay)
    cu, cuh = pack(lengths)
    h0 = randn(g, 2, H, N, P)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, cu, cuh, softplus=False, h0=h0)
    ro, rh = ref.scan(x.double(), dt.double(), A.double(), B.double(), C.double(), None, lengths, h0.double())
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("lengths,mean", [([32, 7], 3.0), ([512], 1.0), ([512], 3.0), ([300, 40, 129], 3.0), ([3000], 3.0)])
def test_ssm_prompt_state_sums_that_cancel(gdr, lengths, mean):
    # The state's rows share a large part that C is orthogonal to, so that an output is a small sum of large
    # terms: an operand of the sum rounded to n bits is off by 2^-n of |C| |S|, some 30 times the output at a mean
    # of 3. The bounds of the outputs' own type hold all the same, in chunks as token by token.
    g, P, N, H, n, T = gen(31), 64, 128, 2, len(lengths), sum(lengths)
    x, dt, A, B, C, _, bias = scan_inputs(g, T, H, P, 1, N, F32)
    B = (mean + randn(g, T, 1, N)).to(BF16)
    half = randn(g, T, 1, N // 2, dtype=BF16)
    C = torch.cat([half, -half], -1)
    h0 = 10 * mean + randn(g, n, H, N, P)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *pack(lengths), dt_bias=bias, h0=h0)
    act = torch.nn.functional.softplus(dt.double() + bias.double())
    ro, rh = ref.scan(x.double(), act, A.double(), B.double(), C.double(), None, lengths, h0.double())
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("lengths", [[32, 7], [512, 100], [3000]])
def test_ssm_prompt_token_sums_that_cancel(gdr, lengths):
    # x changes its sign from token to token under a slow decay: the sum over a chunk's tokens leaves a
    # fraction of its terms
    g, P, N, H, T = gen(32), 64, 128, 2, sum(lengths)
    x, _, A, B, C, _, _ = scan_inputs(g, T, H, P, 1, N, F32)
    sign = 1 - 2 * (torch.arange(T, device="cuda") % 2)
    x = ((8 + 0.25 * randn(g, T, H, P)) * sign[:, None, None]).to(BF16)
    B, C = ((1 + 0.05 * randn(g, T, 1, N)).to(BF16) for _ in range(2))
    dt, A = torch.full((T, H), 0.0625, device="cuda"), torch.full_like(A, -0.01)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *pack(lengths), softplus=False)
    ro, rh = ref.scan(x.double(), dt.double(), A.double(), B.double(), C.double(), None, lengths, None)
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("decay,slow,reset", [(-64.0, 0.01, 1e3), (-1e4, 1e-4, 1e3), (-1.0, 0.02, 1e9)])
def test_ssm_prompt_resets(gdr, decay, slow, reset):
    # tokens whose decay leaves nothing of the state, among slow ones: the decays between the others keep theirs
    g, lengths, H, P, N = gen(33), [300, 128, 20], 2, 64, 128
    T = sum(lengths)
    x, _, A, B, C, _, _ = scan_inputs(g, T, H, P, 1, N, F32)
    dt = torch.where(rand(g, T, H) < 0.05, reset, slow) * (0.5 + rand(g, T, H))
    x = torch.where(dt[:, :, None] > 0.5 * reset - 1, x / reset, x).to(BF16)  # (their terms as large as the others')
    A = torch.full_like(A, decay)
    out, ht = gdr.ssm_fwd(x, dt, A, B, C, *pack(lengths), softplus=False)
    torch.cuda.synchronize()
    gdr.gdr_check_device()
    ro, rh = ref.scan(x.double(), dt.double(), A.double(), B.double(), C.double(), None, lengths, None)
    check(out, ro, "out")
    check(ht, rh, "ht")


@pytest.mark.parametrize("batch,H,P,G,N,dt_dtype,pad,odd", [
    (1, 16, 64, 1, 128, BF16, 0, False), (7, 6, 40, 2, 24, F32, 8, False), (5, 3, 33, 1, 17, BF16, 3, True),
    (2, 2, 256, 1, 256, F32, 0, False), (130, 8, 64, 8, 128, BF16, 64, False), (3, 1, 1, 1, 1, F32, 0, False)])
def test_ssm_step(gdr, batch, H, P, G, N, dt_dtype, pad, odd):
    g, S = gen(batch + P), batch + 2
    state = randn(g, S, H, N, P)
    slots = torch.randperm(S, generator=g, device="cuda")[:batch].to(torch.int32)
    if batch > 2:
        slots[0], slots[2] = S + 5, -1
    live = (slots >= 0) & (slots < S)
    before = state.clone()
    r = before.double()[torch.where(live, slots, 0).long()]
    for step in range(3):
        x, dt, A, B, C, D, bias = scan_inputs(g, batch, H, P, G, N, dt_dtype, pad, odd)
        out = gdr.ssm_step(x, dt, A, B, C, state, D=D, dt_bias=bias, slots=slots, out=full((batch, H, P), BF16))
        act = torch.nn.functional.softplus(dt.double() + bias.double(), threshold=100.0)
        rows = [ref.scan(x[i:i + 1].double(), act[i:i + 1], A.double(), B[i:i + 1].double(), C[i:i + 1].double(),
                         D.double(), [1], r[i:i + 1]) for i in range(batch)]
        ro, r = torch.cat([o for o, _ in rows]), torch.cat([s for _, s in rows])
        check(out, torch.where(live[:, None, None], ro, torch.zeros_like(ro)), f"step {step}")
    used = slots[live].long()
    check(state[used], r[live], "state")
    rest = torch.ones(S, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(state[rest], before[rest])


# ---------------------------------------------------------------------------
# One token of the gated delta rule
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("variant,B,Hqk,HV,l2", [
    ("kda", 1, 4, 4, False), ("kda", 9, 3, 3, True), ("gdn", 1, 1, 3, False), ("gdn", 6, 2, 6, True), ("gdn", 40, 16, 48, True)])
def test_delta_step(gdr, variant, B, Hqk, HV, l2):
    g, S, scale = gen(B + HV), B + 3, 128 ** -0.5
    state = 0.1 * randn(g, S, HV, 128, 128)
    slots = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    if B > 2:
        slots[2] = -7
    live = (slots >= 0) & (slots < S)
    before = state.clone()
    r = before.double()[torch.where(live, slots, 0).long()]
    for step in range(3):
        q, k = randn(g, B, Hqk, 128), randn(g, B, Hqk, 128)
        if not l2:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        q, k, v = q.to(BF16), k.to(BF16), randn(g, B, HV, 128, dtype=BF16)
        gate = -5 * (rand(g, B, HV, 128) if variant == "kda" else rand(g, B, HV))
        if step == 1:
            gate[0, 0] = float("-inf")  # a full reset
        beta = rand(g, B, HV).to(BF16 if variant == "kda" else F32)
        fn = gdr.kda_step if variant == "kda" else gdr.gdn_step
        out = fn(q, k, v, gate, beta, state, scale, slots=slots, out=full((B, HV, 128), BF16), qk_l2norm=l2)
        qh, kh = (t.double().repeat_interleave(HV // Hqk, 1) for t in (q, k))
        ro, r = ref.delta(qh, kh, v.double(), gate.double(), beta.double(), r, scale, l2)
        check(out, torch.where(live[:, None, None], ro, torch.zeros_like(ro)), f"step {step}")
    used = slots[live].long()
    check(state[used], r[live], "state")
    rest = torch.ones(S, dtype=torch.bool, device="cuda")
    rest[used] = False
    assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("variant,Hqk,HV", [("kda", 2, 2), ("gdn", 1, 2)])
def test_delta_steps_continue_a_forward(gdr, variant, Hqk, HV):
    # the end state of a prompt, served token by token, gives the forward's outputs on the whole text
    import synth
    T, cut, scale = 90, 70, 128 ** -0.5
    x = {k: v.cuda() for k, v in synth.make_inputs(variant, T, Hqk, HV, 128, seed=4).items()}
    fwd, step = (gdr.kda_fwd, gdr.kda_step) if variant == "kda" else (gdr.gdn_fwd, gdr.gdn_step)
    names = ("q", "k", "v", "g", "beta")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    whole, end, _ = fwd(*(x[n] for n in names), cu, [0, T], scale, save_for_bwd=False)
    cu2 = torch.tensor([0, cut], dtype=torch.int32, device="cuda")
    _, state, _ = fwd(*(x[n][:cut].contiguous() for n in names), cu2, [0, cut], scale, save_for_bwd=False)
    outs = [step(*(x[n][t:t + 1].contiguous() for n in names), state, scale) for t in range(cut, T)]
    # the forward's own tolerance: its products run on 11-bit operands
    assert rel(torch.cat(outs), whole[cut:]) <= 3e-3 * 2 ** 0.5
    assert rel(state, end) <= 3e-3


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------
NORM = [
    # shape, dtype, post, gate act, residual, pre, fp32 weights, strided, alpha
    ((5, 3, 128), BF16, True, "silu", False, False, False, True, 1.0),
    ((7, 48, 128), BF16, True, "sigmoid", False, False, True, False, 1.0),
    ((33, 64), F16, True, "silu", False, False, False, False, 1.0),
    ((9, 2048), BF16, True, None, True, True, False, False, 0.5),
    ((1, 2048), BF16, False, None, True, True, False, False, 1.0),
    ((130, 1000), F32, True, "silu", True, True, False, False, 0.25),
    ((6, 1, 4096), BF16, False, None, False, True, True, False, 1.0),
    ((3, 8192), F32, True, None, True, True, False, False, 2.0),
    ((4, 16384), BF16, True, "silu", True, True, False, False, 0.5),
    ((2, 16384), F32, True, "sigmoid", True, True, False, False, 0.5),
    ((3, 16383), BF16, True, "silu", True, True, False, False, 0.5),
    ((11, 37), BF16, True, "silu", True, True, False, True, 0.7),
    ((5, 2, 257), F32, False, "sigmoid", True, True, False, True, 1.5),
    ((3, 1), F32, True, None, True, True, False, False, 1.0),
    ((2000, 16), BF16, True, "silu", False, True, False, False, 1.0),
    ((600, 2, 256), F16, False, None, True, False, False, False, 0.5),
    ((2, 3, 4, 96), BF16, True, "silu", True, True, False, False, 0.5),
    ((128,), BF16, True, None, False, False, False, False, 1.0),
    ((0, 4, 128), BF16, True, "silu", False, False, False, False, 1.0),
    ((5000, 320), BF16, False, None, True, True, False, False, 1.0),
]
# rows of every width class: lanes of a warp, one to four warps, clusters of two to nine blocks (sixteen of FP32);
# lengths that are no whole number of 16-byte pieces, packed one after another or strided
NORM += [((rows, D), dt, True, "silu" if D % 3 else None, True, True, False, False, 0.5) for rows, D, dt in (
    (67, 3, BF16), (130, 17, F16), (41, 31, BF16), (35, 61, F32), (29, 127, BF16), (300, 249, BF16), (23, 511, F16),
    (19, 520, BF16), (17, 1021, BF16), (700, 1032, BF16), (9, 1536, F32), (11, 2047, BF16), (21, 2056, BF16),
    (10, 2050, F32), (13, 4097, BF16), (33, 5120, BF16), (3, 6144, F32), (5, 7168, F16), (9, 12289, BF16),
    (2, 16381, F32), (4, 10246, F32))]
NORM += [((43, 3, 77), BF16, True, "sigmoid", False, False, True, False, 1.0), ((1000, 5), F32, False, None, True, True, False, False, 1.0),
         ((7, 3001), BF16, True, "silu", True, True, False, True, 0.5), ((5, 9001), F32, True, None, True, True, True, True, 0.5)]


@pytest.mark.parametrize("shape,dtype,post,act,residual,pre,wf32,odd,alpha", NORM)
def test_norm_forward_and_gradients(gdr, shape, dtype, post, act, residual, pre, wf32, odd, alpha):
    g, D, wt = gen(shape[-1] + len(shape)), shape[-1], F32 if wf32 else dtype

    def rows(scale=1.0):
        t = (scale * randn(g, *shape)).to(dtype)
        if not odd:
            return t
        wide = torch.full((*shape[:-1], D + 3), 9.0, dtype=dtype, device="cuda")
        wide[..., 1:1 + D] = t
        return wide[..., 1:1 + D]
    x, z, r = rows(), rows() if act else None, rows(2.0) if residual else None
    wp = (1 + 0.2 * randn(g, D)).to(wt) if post else None
    w = (1 + 0.2 * randn(g, D)).to(wt) if pre else None
    has_h = residual or not pre
    dh, dy = rows() if has_h else None, rows() if pre else None
    args = dict(weight=w, post_weight=wp, gate=z, act=act or "silu", residual=r, res_scale=alpha, eps=1e-5)
    h, y = gdr.norm_fwd(x, **args, h=full(shape, dtype) if has_h else None, y=full(shape, dtype) if pre else None)
    leaves = {k: t.double().requires_grad_() for k, t in
              (("x", x), ("w", w), ("wp", wp), ("z", z), ("r", r)) if t is not None}
    rh, ry = ref.norms(leaves["x"], leaves.get("w"), leaves.get("wp"), leaves.get("z"), act, leaves.get("r"), alpha, 1e-5)
    assert (h is None) == (not has_h) and (y is None) == (not pre)
    if has_h:
        check(h, rh, "h")
    if pre:
        check(y, ry, "y")
    total = (rh * dh.double()).sum() if has_h else 0
    total = total + (ry * dy.double()).sum() if pre else total
    names = {"x": "dx", "w": "dweight", "wp": "dpost_weight", "z": "dgate", "r": "dresidual"}
    rg = dict(zip((names[k] for k in leaves), torch.autograd.grad(total, list(leaves.values()))))
    bufs = {k: full(v.shape, F32 if "weight" in k else dtype) for k, v in rg.items()}
    got = gdr.norm_bwd(x, **args, dh=dh, dy=dy, grads=bufs)
    assert {k for k, v in got.items() if v is not None} == set(rg)
    for k, v in rg.items():
        check(got[k], v, k)
    again = gdr.norm_bwd(x, **args, dh=dh, dy=dy)
    for k in rg:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("D", [7, 129, 1021, 4099])
def test_norm_rows_keep_to_themselves(gdr, D):
    # rows whose pieces of 16 bytes reach into the rows beside them: a row of NaN and one of infinities stay alone
    g = gen(D)
    x, r, dy = (randn(g, 24, D, dtype=BF16) for _ in range(3))
    w = (1 + 0.2 * randn(g, D)).to(BF16)
    bad = x.clone()
    bad[5], bad[18] = float("nan"), float("inf")
    keep = [i for i in range(24) if i not in (5, 18)]
    h, y = gdr.norm_fwd(x, weight=w, post_weight=w, residual=r)
    h2, y2 = gdr.norm_fwd(bad, weight=w, post_weight=w, residual=r)
    assert torch.equal(h[keep], h2[keep]) and torch.equal(y[keep], y2[keep])
    a = gdr.norm_bwd(x, weight=w, post_weight=w, residual=r, dh=dy, dy=dy)
    b = gdr.norm_bwd(bad, weight=w, post_weight=w, residual=r, dh=dy, dy=dy)
    assert torch.equal(a["dx"][keep], b["dx"][keep]) and torch.equal(a["dresidual"][keep], b["dresidual"][keep])
    assert torch.isnan(b["dx"][5]).all()


@pytest.mark.parametrize("widths", [(2047, 3000), (3000, 2047, 3064), (2045, 2056), (1024, 2048, 2049, 4096), (4099, 9001, 16384)])
def test_norm_partial_rows_stay_in_the_workspace(gdr, widths):
    # widths that share a kernel, but not the number of partial rows their workspaces hold, one after another
    g = gen(35)
    for D in widths:
        rows, need = 4000, gdr.norm_workspace_bytes(D)
        x, r, dy = (randn(g, rows, D, dtype=BF16) for _ in range(3))
        w = (1 + 0.1 * randn(g, D)).to(BF16)
        buf = torch.full((need + 4096 * D,), 0x5a, dtype=torch.uint8, device="cuda")
        got = gdr.norm_bwd(x, weight=w, post_weight=w, residual=r, dy=dy, scratch=buf[:need])
        assert bool((buf[need:] == 0x5a).all()), D
        a = [t.double().requires_grad_() for t in (x, w, w, r)]
        torch.autograd.backward(ref.norms(a[0], a[1], a[2], None, "silu", a[3], 1.0, 1e-6)[1], dy.double())
        check(got["dx"], a[0].grad, f"dx {D}")
        check(got["dweight"], a[1].grad, f"dweight {D}")
        check(got["dpost_weight"], a[2].grad, f"dpost_weight {D}")


def test_norm_gradients_by_differences(gdr):
    g, shape = gen(8), (6, 2, 40)
    a = {"x": randn(g, *shape), "gate": randn(g, *shape), "residual": randn(g, *shape), "weight": 1 + 0.3 * randn(g, 40),
         "post_weight": 1 + 0.3 * randn(g, 40)}
    dh, dy = randn(g, *shape), randn(g, *shape)

    def loss(t):
        h, y = gdr.norm_fwd(**t, res_scale=0.5)
        return float((h.double() * dh.double()).sum() + (y.double() * dy.double()).sum())

    got = gdr.norm_bwd(**a, res_scale=0.5, dh=dh, dy=dy)
    for name in a:
        v, eps = randn(g, *a[name].shape), 1e-2
        diff = (loss({**a, name: a[name] + eps * v}) - loss({**a, name: a[name] - eps * v})) / (2 * eps)
        grad = got["d" + name].double()
        inner = float((grad * v.double()).sum())
        assert abs(diff - inner) <= 2e-3 * float(grad.norm() * v.double().norm()) + 1e-2, (name, diff, inner)


def test_norm_rows_of_zeros_and_of_one_gradient(gdr):
    # a row of zeros divides by sqrt(eps) only; dh without dy; -inf gates close
    x = torch.zeros(3, 128, device="cuda", dtype=BF16)
    x[1] = 1.0
    w = torch.ones(128, device="cuda", dtype=BF16)
    z = torch.full_like(x, float("-inf"))
    h, _ = gdr.norm_fwd(x, post_weight=w)
    assert torch.equal(h[0], x[0]) and torch.isfinite(h).all()
    h, _ = gdr.norm_fwd(x, post_weight=w, gate=z)
    assert torch.equal(h, torch.zeros_like(h))
    g = gdr.norm_bwd(x, post_weight=w, gate=z, dh=torch.ones_like(x))
    assert all(torch.isfinite(t.float()).all() for t in g.values())
    r = torch.ones_like(x)
    g = gdr.norm_bwd(x, weight=w, residual=r, dh=r)
    assert g["dx"] is g["dresidual"] and torch.equal(g["dx"], r) and torch.equal(g["dweight"], torch.zeros(128, device="cuda"))


# ---------------------------------------------------------------------------
# Streams and refusals
# ---------------------------------------------------------------------------
def test_calls_run_on_the_stream_they_are_given(gdr):
    g, lengths = gen(9), [500, 13]
    cu, cuh = pack(lengths)
    x, w = randn(g, 513, 256, dtype=BF16), randn(g, 256, 4, dtype=BF16)
    want, _ = gdr.sconv_fwd(x, w, None, cu, cuh)
    h, _ = gdr.norm_fwd(x, post_weight=w[:, 0].contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = gdr.sconv_fwd(x, w, None, cu, cuh, stream=s)
    h2, _ = gdr.norm_fwd(out, post_weight=w[:, 0].contiguous(), stream=s)  # ordered after the line above
    s.synchronize()
    assert torch.equal(out, want)
    ref_h, _ = gdr.norm_fwd(want, post_weight=w[:, 0].contiguous())
    assert torch.equal(h2, ref_h)


def test_calls_are_captured_in_a_graph(gdr):
    g, B = gen(10), 3
    x, w = randn(g, B, 128, dtype=BF16), randn(g, 128, 4, dtype=BF16)
    state, eager = (torch.zeros(B, 3, 128, device="cuda", dtype=BF16) for _ in range(2))
    gdr.sconv_step(x, w, None, eager)
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gdr.sconv_step(x, w, None, torch.zeros_like(state), out=out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdr.sconv_step(x, w, None, state, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(state, eager)


def test_calls_of_several_kernels_are_captured_in_a_graph(gdr):
    # calls whose own kernels overlap by programmatic launches: a prompt in segments and in one, the convolution's and
    # the norms' gradients; replayed on new inputs they give what the calls give
    g, lengths, H, P, N, C = gen(15), [3000, 70], 2, 64, 128, 256
    T = sum(lengths)
    cu, cuh = pack(lengths)
    xs, dt, A, B, Cm, D, bias = scan_inputs(g, T, H, P, 1, N, F32)
    x, dy, w = randn(g, T, C, dtype=BF16), randn(g, T, C, dtype=BF16), randn(g, C, 4, dtype=BF16)
    nw = (1 + 0.1 * randn(g, C)).to(BF16)

    def calls():
        out, ht = gdr.ssm_fwd(xs, dt, A, B, Cm, cu, cuh, D=D, dt_bias=bias)
        conv = gdr.sconv_bwd(x, w, None, cu, cuh, dy)
        norm = gdr.norm_bwd(x, weight=nw, post_weight=nw, residual=dy, dy=dy)
        return [out, ht, conv["dx"], conv["dweight"], norm["dx"], norm["dresidual"], norm["dweight"], norm["dpost_weight"]]
    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for seed in (16, 17):
        h = gen(seed)
        for t in (xs, dt, x, dy):
            t.copy_(0.5 * randn(h, *t.shape))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(captured, calls())):
            assert torch.equal(a, b), i
    gdr.gdr_check_device()


def test_calls_from_several_threads(gdr):
    # the interpreter's lock is released during a call: widths that share kernels, each thread on a stream of its own
    import threading
    g = gen(18)
    inputs = [[randn(g, 700, D, dtype=BF16) for _ in range(2)] + [(1 + 0.1 * randn(g, D)).to(BF16)] for D in (2047, 3000, 2048, 66)]
    want = [gdr.norm_bwd(x, weight=w, post_weight=w, residual=r, dy=r) for x, r, w in inputs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            x, r, w = inputs[i]
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(30):
                    got = gdr.norm_bwd(x, weight=w, post_weight=w, residual=r, dy=r)
                stream.synchronize()
                failed.extend((i, k) for k in got if not torch.equal(got[k], want[i][k]))
        except Exception as e:  # a thread's exception would be lost
            failed.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(inputs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_refusals(gdr):
    g = gen(11)
    x, w = randn(g, 10, 16, dtype=BF16), randn(g, 16, 4, dtype=BF16)
    cu, cuh = pack([10])
    bad = [
        lambda: gdr.sconv_fwd(x, w[:, :1].contiguous(), None, cu, cuh),  # one tap
        lambda: gdr.sconv_fwd(x, w.half(), None, cu, cuh),  # weights of another type
        lambda: gdr.sconv_fwd(x.double(), w.double(), None, cu, cuh),
        lambda: gdr.sconv_fwd(x, w, None, cu, [0, 9]),  # cu[N] != T
        lambda: gdr.sconv_fwd(x, w, None, cu.long(), cuh),
        lambda: gdr.sconv_fwd(x.cpu(), w, None, cu, cuh),
        lambda: gdr.sconv_fwd(x, w.cpu(), None, cu, cuh),
        lambda: gdr.sconv_fwd(x.t(), w, None, cu, cuh),  # rows not dense
        lambda: gdr.sconv_fwd(x, w, None, cu, cuh, s0=torch.zeros(1, 4, 16, device="cuda", dtype=BF16)),
        lambda: gdr.sconv_bwd(x, w, None, cu, cuh, x[:9]),
        lambda: gdr.sconv_bwd(x, w, None, cu, cuh, x, scratch=torch.empty(256, dtype=torch.uint8, device="cuda")),
        lambda: gdr.sconv_step(x, w, None, torch.zeros(9, 3, 16, device="cuda", dtype=BF16)),  # fewer states than rows
        lambda: gdr.norm_fwd(x),  # nothing to do
        lambda: gdr.norm_fwd(x, weight=w[:, 0]),  # a strided weight
        lambda: gdr.norm_fwd(x, weight=torch.ones(16, device="cuda", dtype=BF16), act="gelu"),
        lambda: gdr.norm_bwd(x, post_weight=torch.ones(16, device="cuda", dtype=BF16)),  # no gradient
        lambda: gdr.norm_bwd(x, post_weight=torch.ones(16, device="cuda", dtype=BF16), dy=x),
    ]
    xs, dt, A, B, C, D, bias = scan_inputs(g, 10, 4, 64, 2, 128, F32)
    bad += [
        lambda: gdr.ssm_fwd(xs, dt[:, :3], A, B, C, cu, cuh),
        lambda: gdr.ssm_fwd(xs, dt, A, B, C[..., :64], cu, cuh),
        lambda: gdr.ssm_fwd(xs.float(), dt, A, B, C, cu, cuh),
        lambda: gdr.ssm_fwd(xs[:, :3], dt[:, :3], A[:3], B, C, cu, cuh),  # 3 heads, 2 groups
        lambda: gdr.ssm_fwd(xs, dt, A.double(), B, C, cu, cuh),
        lambda: gdr.ssm_fwd(xs, dt, A, B, C, cu, [0, 11]),
        lambda: gdr.ssm_step(xs, dt, A, B, C, torch.zeros(9, 4, 128, 64, device="cuda")),
        lambda: gdr.ssm_step(xs, dt, A, B, C, torch.zeros(10, 4, 64, 128, device="cuda")),
    ]
    q = randn(g, 2, 2, 128, dtype=BF16)
    gate, beta = torch.zeros(2, 2, device="cuda"), torch.zeros(2, 2, device="cuda")
    st = torch.zeros(2, 2, 128, 128, device="cuda")
    bad += [
        lambda: gdr.gdn_step(q, q, q, gate, beta, st[:1], 1.0),
        lambda: gdr.gdn_step(q, q, q, gate, beta.to(BF16), st, 1.0),
        lambda: gdr.kda_step(q, q, q, gate, beta.to(BF16), st, 1.0),  # KDA's gate is per channel
        lambda: gdr.gdn_step(q[..., :64], q[..., :64], q[..., :64], gate, beta, st, 1.0),
        lambda: gdr.gdn_step(q, q, q, gate, beta, st, 1.0, slots=torch.zeros(2, device="cuda", dtype=torch.int64)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()


def test_refuses_sizes_past_32_bits(gdr):
    # (no memory behind them: every row is the same one)
    x = torch.ones(1, device="cuda", dtype=BF16).expand(1, 2**32 + 4, 1)
    w = torch.ones(1, device="cuda", dtype=BF16)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.norm_fwd(x, post_weight=w)
    with pytest.raises(ValueError, match="2\\^31"):
        gdr.norm_bwd(x, post_weight=w, dh=x)


def test_binding_holds_nothing(gdr):
    # references and device memory after calls, refused calls included, are what they were before
    import sys
    g = gen(14)
    x, w, r = randn(g, 40, 64, dtype=BF16), randn(g, 64, 4, dtype=BF16), randn(g, 64, dtype=BF16)
    cu, cuh = pack([30, 10])
    bufs = {"dx": torch.empty_like(x)}

    def calls():
        out, st = gdr.sconv_fwd(x, w, None, cu, cuh, s0=None)
        grads = gdr.sconv_bwd(x, w, None, cu, cuh, out, grads=bufs)
        assert grads["dx"] is bufs["dx"] and grads["dbias"] is None and list(bufs) == ["dx"]
        h, y = gdr.norm_fwd(x, weight=r, residual=out)
        gdr.norm_bwd(x, weight=r, residual=out, dh=h, dy=y)
        for bad in (lambda: gdr.sconv_fwd(x, w, None, cu, [0, 30, 41]), lambda: gdr.sconv_fwd(x, w, r[1:], cu, cuh),
                    lambda: gdr.sconv_bwd(x, w, None, cu, cuh, out, grads={"dx": r}), lambda: gdr.norm_fwd(x, weight="r"),
                    lambda: gdr.sconv_fwd(x, w, None, cu, cuh, out=x)):
            with pytest.raises(ValueError):
                bad()
        gdr.sconv_fwd(x, w, None, cu, [0, 30, 40])  # any sequence of whole numbers
    calls()
    held = (x, w, r, cu, bufs["dx"])
    before = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    assert ([sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()) == before
