"""The operators around the gated delta rule, as measured: cases, inputs, plain forms and 64-bit values.

Four families, each in the forms a program runs them in:

* sconv: the short causal depthwise convolution over packed documents (prompt: forward with start and end
  states; train: forward and backward; step: one token of each sequence against a rolling state);
* ssm: the selective state space scan with a scalar decay a head (prompt, step);
* kda / gdn: one token of the gated delta rule a sequence, the state updated in place;
* norm: the norm after a block, its gate, the scaled residual and the norm before the next block (fwd, train).

A case is a dict of plain values; `lengths` lists document lengths.  `own` false computes the plain forms
(elementary torch operations in 32 bits, rounded once at the end), true calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
D = 128  # head dimension of the gated delta rule


def listed():
    return [
        # One sequence decoding through a KDA layer of 4 heads: q, k and v's channels, latency alone.
        {"name": "sconv_step_b1", "op": "sconv", "mode": "step", "batch": 1, "C": 1536, "W": 4, "dtype": "bf16",
         "bias": False, "silu": True},
        # A ragged batch of prompts through a KDA layer of 16 heads, continued from and into cached states.
        {"name": "sconv_prompt_ragged", "op": "sconv", "mode": "prompt", "lengths": "1,129,0,2047,63,1000,3,858",
         "C": 6144, "W": 4, "dtype": "bf16", "bias": True, "silu": True},
        # Training on one document through the convolution of a grouped GDN layer (16, 48).
        {"name": "sconv_train_gdn_1doc", "op": "sconv", "mode": "train", "lengths": "32768", "C": 10240, "W": 4,
         "dtype": "bf16", "bias": False, "silu": True},
        # One sequence decoding through a scan layer: latency alone.
        {"name": "ssm_step_b1", "op": "ssm", "mode": "step", "batch": 1, "H": 16, "P": 64, "G": 1, "N": 128,
         "dt": "bf16"},
        # A served batch of sequences decoding through a wide scan layer.
        {"name": "ssm_step_b256", "op": "ssm", "mode": "step", "batch": 256, "H": 64, "P": 64, "G": 8, "N": 128,
         "dt": "bf16"},
        # Short prompts of odd lengths, one of them empty, continued from cached states.
        {"name": "ssm_prompt_ragged", "op": "ssm", "mode": "prompt", "lengths": "1,63,64,0,65,129,300", "H": 16,
         "P": 64, "G": 1, "N": 128, "dt": "f32", "h0": True},
        # One long prompt.
        {"name": "ssm_prompt_32k", "op": "ssm", "mode": "prompt", "lengths": "32768", "H": 64, "P": 64, "G": 8,
         "N": 128, "dt": "bf16", "h0": False},
        # One sequence decoding through a KDA layer of 4 heads: latency alone.
        {"name": "kda_step_b1", "op": "kda", "batch": 1, "Hqk": 4, "HV": 4, "l2": False},
        # A served batch decoding through a grouped GDN layer (16, 48).
        {"name": "gdn_step_b128", "op": "gdn", "batch": 128, "Hqk": 16, "HV": 48, "l2": True},
        # One token of one sequence between two blocks: latency alone.
        {"name": "norm_block_b1", "op": "norm", "mode": "fwd", "rows": 1, "heads": 1, "D": 2048, "dtype": "bf16",
         "post": True, "gate": "", "residual": True, "pre": True},
        # A ragged prompt between two blocks: norm after, residual scale, residual, norm before.
        {"name": "norm_block_train", "op": "norm", "mode": "train", "rows": 8191, "heads": 1, "D": 2048,
         "dtype": "bf16", "post": True, "gate": "", "residual": True, "pre": True},
        # Training through the gated output norm of a grouped GDN layer, 48 heads of 128.
        {"name": "norm_gate_train", "op": "norm", "mode": "train", "rows": 32768, "heads": 48, "D": 128,
         "dtype": "bf16", "post": True, "gate": "silu", "residual": False, "pre": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cut(rng, total):
    """`total` tokens in 1 to 8 documents at random cuts (some may be empty)."""
    n = rng.randint(1, 8)
    cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
    edges = [0] + cuts + [total]
    return ",".join(str(b - a) for a, b in zip(edges, edges[1:]))


def draw(rng):
    op = rng.choice(["sconv", "ssm", "ssm", "delta", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "sconv":
        mode = rng.choice(["step", "prompt", "train"])
        C = _log_int(rng, 8, 10240)
        case = {"op": "sconv", "mode": mode, "C": C if rng.random() < 0.4 else -(-C // 8) * 8, "W": rng.randint(2, 4),
                "dtype": dtype, "bias": rng.random() < 0.5, "silu": rng.random() < 0.8}
        if mode == "step":
            case["batch"] = _log_int(rng, 1, 512)
        else:
            case["lengths"] = _cut(rng, _log_int(rng, 1, 16384 if dtype == "f32" else 32768))
        return case
    if op == "ssm":
        G = rng.choice([1, 1, 2, 4, 8])
        case = {"op": "ssm", "mode": rng.choice(["step", "prompt", "prompt"]), "H": G * rng.randint(1, 64 // G),
                "P": rng.choice([32, 64, 64, 128]), "G": G, "N": rng.choice([16, 64, 128, 128]),
                "dt": rng.choice(["bf16", "f32"])}
        if case["mode"] == "step":
            case["batch"] = _log_int(rng, 1, 256)
        else:
            case["lengths"] = _cut(rng, _log_int(rng, 1, 32768 * 64 * 64 // max(64 * 64, case["H"] * case["P"])))
            case["h0"] = rng.random() < 0.5
        return case
    if op == "delta":
        Hqk = rng.choice([1, 2, 4, 8, 16])
        variant = rng.choice(["kda", "gdn"])
        return {"op": variant, "batch": _log_int(rng, 1, 128), "Hqk": Hqk,
                "HV": Hqk if variant == "kda" else Hqk * rng.randint(1, 3), "l2": rng.random() < 0.5}
    heads = rng.choice([1, 1, 4, 16, 48])
    width = _log_int(rng, 16, 8192) if heads == 1 else rng.choice([64, 128, 256])
    if heads == 1 and rng.random() < 0.6:
        width = -(-width // 8) * 8
    kind = rng.choice(["gate", "block", "pre"])
    return {"op": "norm", "mode": rng.choice(["fwd", "train"]), "rows": _log_int(rng, 1, min(32768, (1 << 26) // (heads * width))),
            "heads": heads, "D": width, "dtype": dtype, "post": kind != "pre",
            "gate": rng.choice(["silu", "sigmoid"]) if kind == "gate" else rng.choice(["", "silu"]),
            "residual": kind != "gate", "pre": kind != "gate"}


def _lengths(case):
    return [int(n) for n in case["lengths"].split(",")]


def work(case):
    op, mode = case["op"], case.get("mode")
    if op == "sconv":
        e, C, W = BYTES[case["dtype"]], case["C"], case["W"]
        if mode == "step":
            return {"bytes": case["batch"] * C * e * (2 + 2 * (W - 1)) + 4 * C * W, "flops": 2.0 * case["batch"] * C * W}
        lens = _lengths(case)
        tc = sum(lens) * C
        if mode == "prompt":
            return {"bytes": 2 * tc * e + 2 * len(lens) * (W - 1) * C * e + 4 * C * W, "flops": 2.0 * tc * W}
        # forward: x in, y out; backward: x and dy in, dx out
        return {"bytes": 5 * tc * e + 8 * C * W, "flops": 8.0 * tc * W}
    if op == "ssm":
        H, P, G, N = case["H"], case["P"], case["G"], case["N"]
        if mode == "step":
            b = case["batch"]
            return {"bytes": b * (8.0 * H * N * P + 4 * H * P + 4 * G * N + 4 * H), "flops": 5.0 * b * H * N * P}
        lens = _lengths(case)
        T = sum(lens)
        states = len(lens) * H * N * P * 4 * (2 if case["h0"] else 1)
        # the recurrence: decay, outer product and read-out of the state for each token
        return {"bytes": T * (4 * H * P + 4 * G * N + BYTES[case["dt"]] * H) + states, "flops": 5.0 * T * H * N * P}
    if op in ("kda", "gdn"):
        b, Hqk, HV = case["batch"], case["Hqk"], case["HV"]
        gates = HV * (4 * D + 2) if op == "kda" else HV * 8
        return {"bytes": b * (HV * D * D * 8.0 + 4 * Hqk * D + 4 * HV * D + gates), "flops": 7.0 * b * HV * D * D}
    n, e = case["rows"] * case["heads"] * case["D"], BYTES[case["dtype"]]
    gate, res, pre = bool(case["gate"]), case["residual"], case["pre"]
    fwd_in = 1 + gate + res
    fwd_out = (1 if res or not pre else 0) + pre
    moved = fwd_in + fwd_out
    if mode == "train":
        moved += fwd_in + fwd_out + fwd_in  # the inputs again, the outputs' gradients, the inputs' gradients
    return {"bytes": n * e * moved, "flops": n * (10.0 if mode == "fwd" else 40.0)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pack(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "sconv":
        t, C, W = DTYPES[case["dtype"]], case["C"], case["W"]
        s["weight"] = ((_rand(g, C, W) * 2 - 1) * W ** -0.5).to(t)
        s["b"] = (0.1 * _randn(g, C)).to(t) if case["bias"] else None
        if case["mode"] == "step":
            n = case["batch"]
            s["x"] = _randn(g, n, C).to(t)
            s["state"] = _randn(g, n + 3, W - 1, C).to(t)  # a pool with free slots
            s["slots"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)
            return s
        lens = _lengths(case)
        s["cu_host"], s["cu"] = _pack(lens)
        s["x"] = _randn(g, sum(lens), C).to(t)
        if case["mode"] == "train":
            s["dout"] = _randn(g, sum(lens), C).to(t)
        else:
            s["s0"] = _randn(g, len(lens), W - 1, C).to(t)
        return s
    if op == "ssm":
        H, P, G, N = case["H"], case["P"], case["G"], case["N"]
        step = case["mode"] == "step"
        lens = None if step else _lengths(case)
        T = case["batch"] if step else sum(lens)
        # x, B and C are slices of the convolution's output, as a layer hands them over
        xbc = torch.nn.functional.silu(_randn(g, T, H * P + 2 * G * N)).to(torch.bfloat16)
        s["x"] = xbc[:, : H * P].unflatten(1, (H, P))
        s["B"] = xbc[:, H * P: H * P + G * N].unflatten(1, (G, N))
        s["C"] = xbc[:, H * P + G * N:].unflatten(1, (G, N))
        s["dtr"] = _randn(g, T, H).to(DTYPES[case["dt"]])
        s["A"] = -(1 + 15 * _rand(g, H))
        dt0 = torch.exp(math.log(1e-3) + _rand(g, H) * (math.log(0.1) - math.log(1e-3)))
        s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))  # softplus of it is dt0
        s["Dskip"] = 1 + 0.1 * _randn(g, H)
        if step:
            s["state"] = 0.3 * _randn(g, T + 3, H, N, P)
            s["slots"] = torch.randperm(T + 3, generator=g, device="cuda")[:T].to(torch.int32)
        else:
            s["cu_host"], s["cu"] = _pack(lens)
            s["s0"] = 0.3 * _randn(g, len(lens), H, N, P) if case["h0"] else None
        return s
    if op in ("kda", "gdn"):
        n, Hqk, HV = case["batch"], case["Hqk"], case["HV"]
        q, k = _randn(g, n, Hqk, D), _randn(g, n, Hqk, D)
        if not case["l2"]:
            q, k = q / q.norm(dim=-1, keepdim=True), k / k.norm(dim=-1, keepdim=True)
        s["q"], s["k"] = q.to(torch.bfloat16), k.to(torch.bfloat16)
        s["v"] = _randn(g, n, HV, D).to(torch.bfloat16)
        s["g"] = -5 * (_rand(g, n, HV, D) if op == "kda" else _rand(g, n, HV))
        s["beta"] = _rand(g, n, HV).to(torch.bfloat16 if op == "kda" else torch.float32)
        s["state"] = 0.05 * _randn(g, n + 3, HV, D, D)
        s["slots"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)
        return s
    t, shape = DTYPES[case["dtype"]], (case["rows"], case["heads"], case["D"])
    s["x"] = _randn(g, *shape).to(t)
    s["z"] = _randn(g, *shape).to(t) if case["gate"] else None
    s["r"] = (2 * _randn(g, *shape)).to(t) if case["residual"] else None
    s["w_post"] = (1 + 0.1 * _randn(g, case["D"])).to(t) if case["post"] else None
    s["w"] = (1 + 0.1 * _randn(g, case["D"])).to(t) if case["pre"] else None
    s["alpha"] = 0.5 if case["residual"] else 1.0
    if case["mode"] == "train":
        s["dh"] = _randn(g, *shape).to(t) if case["residual"] or not case["pre"] else None
        s["dy"] = _randn(g, *shape).to(t) if case["pre"] else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    op, mode = s["op"], s.get("mode")
    if op == "sconv":
        return _conv_step(s) if mode == "step" else _conv_pack(s)
    if op == "ssm":
        return _ssm_step(s) if mode == "step" else _ssm_prompt(s)
    return _delta_step(s) if op in ("kda", "gdn") else _norm(s)


def _run_own(s):
    import gated_delta_rule_varlen_gb300 as gdr

    op, mode = s["op"], s.get("mode")
    if op == "sconv":
        if mode == "step":
            y = gdr.sconv_step(s["x"], s["weight"], s["b"], s["state"], slots=s["slots"], silu=s["silu"])
            return {"out": y, "state": s["state"]}
        if mode == "prompt":
            y, st = gdr.sconv_fwd(s["x"], s["weight"], s["b"], s["cu"], s["cu_host"], s0=s["s0"], silu=s["silu"])
            return {"out": y, "state": st}
        y, _ = gdr.sconv_fwd(s["x"], s["weight"], s["b"], s["cu"], s["cu_host"], silu=s["silu"], want_st=False)
        grads = gdr.sconv_bwd(s["x"], s["weight"], s["b"], s["cu"], s["cu_host"], s["dout"], silu=s["silu"])
        return {"out": y, **{k: v for k, v in grads.items() if v is not None}}
    if op == "ssm":
        if mode == "step":
            y = gdr.ssm_step(s["x"], s["dtr"], s["A"], s["B"], s["C"], s["state"], D=s["Dskip"], dt_bias=s["dt_bias"],
                             slots=s["slots"])
            return {"out": y, "state": s["state"]}
        y, ht = gdr.ssm_fwd(s["x"], s["dtr"], s["A"], s["B"], s["C"], s["cu"], s["cu_host"], D=s["Dskip"],
                            dt_bias=s["dt_bias"], h0=s["s0"])
        return {"out": y, "state": ht}
    if op in ("kda", "gdn"):
        step = gdr.kda_step if op == "kda" else gdr.gdn_step
        y = step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], D ** -0.5, slots=s["slots"], qk_l2norm=s["l2"])
        return {"out": y, "state": s["state"]}
    args = dict(weight=s["w"], post_weight=s["w_post"], gate=s["z"], act=s["gate"] or "silu", residual=s["r"],
                res_scale=s["alpha"], eps=EPS)
    h, y = gdr.norm_fwd(s["x"], **args)
    got = {"h": h, "y": y}
    if mode == "train":
        got.update(gdr.norm_bwd(s["x"], dh=s["dh"], dy=s["dy"], **args))
    return {k: v for k, v in got.items() if v is not None}


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _act_grad(z):
    """d silu(z) / dz"""
    sg = _sigmoid(z)
    return sg * (1 + z * (1 - sg))


def _conv_pack(s):
    x, w, W, lens = s["x"].float(), s["weight"].float(), s["W"], _lengths(s)
    T, C, n, K = x.shape[0], x.shape[1], len(lens), s["W"] - 1
    cu = s["cu"].long()
    tok = torch.arange(T, device="cuda")
    doc = torch.searchsorted(cu[1:], tok, right=True)
    start, end = cu[doc], cu[doc + 1]
    # rows of `rows`: one of zeros, the start states, the tokens
    s0 = s.get("s0")
    before = x.new_zeros(n * K, C) if s0 is None else s0.float().reshape(n * K, C)
    rows = torch.cat([x.new_zeros(1, C), before, x])
    taps = torch.arange(W, device="cuda")
    at = tok[:, None] - K + taps  # [T, W]
    at = torch.where(at >= start[:, None], 1 + n * K + at, 1 + doc[:, None] * K + (at - start[:, None] + K))
    z = (rows[at] * w.t()).sum(1)
    if s["b"] is not None:
        z = z + s["b"].float()
    y = (z * _sigmoid(z) if s["silu"] else z).to(s["x"].dtype)
    if s["mode"] == "prompt":
        last = cu[1:, None] - K + torch.arange(K, device="cuda")  # [n, K]
        last = torch.where(last >= cu[:-1, None], 1 + n * K + last,
                           1 + torch.arange(n, device="cuda")[:, None] * K + (last - cu[:-1, None] + K))
        return {"out": y, "state": rows[last].to(s["x"].dtype)}
    dz = s["dout"].float()
    if s["silu"]:
        dz = dz * _act_grad(z)
    dw = (rows[at] * dz[:, None, :]).sum(0).t().contiguous()
    to = tok[:, None] + K - taps  # the token that reads this one through tap j
    dzp = torch.cat([dz, dz.new_zeros(1, C)])
    dx = (dzp[torch.where(to < end[:, None], to, T)] * w.t()).sum(1)
    got = {"out": y, "dx": dx.to(s["x"].dtype), "dweight": dw}
    if s["b"] is not None:
        got["dbias"] = dz.sum(0)
    return got


def _conv_step(s):
    slots = s["slots"].long()
    xx = torch.cat([s["state"][slots], s["x"][:, None, :]], 1)  # [n, W, C]
    z = (xx.float() * s["weight"].float().t()).sum(1)
    if s["b"] is not None:
        z = z + s["b"].float()
    s["state"][slots] = xx[:, 1:]
    return {"out": (z * _sigmoid(z) if s["silu"] else z).to(s["x"].dtype), "state": s["state"]}


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-torch.abs(x)))


def _ssm_step(s):
    H, G, slots = s["H"], s["G"], s["slots"].long()
    dt = _softplus(s["dtr"].float() + s["dt_bias"])
    Bh = s["B"].float().repeat_interleave(H // G, 1)
    Ch = s["C"].float().repeat_interleave(H // G, 1)
    x = s["x"].float()
    S = s["state"][slots] * torch.exp(dt * s["A"])[..., None, None] + (dt[..., None] * Bh)[..., None] * x[:, :, None, :]
    s["state"][slots] = S
    y = (S * Ch[..., None]).sum(2) + s["Dskip"][:, None] * x
    return {"out": y.to(s["x"].dtype), "state": s["state"]}


def _ssm_prompt(s, Q=64):
    """Chunks of Q tokens that restart at each document: inside a chunk by the masked product, across chunks by the decays."""
    H, P, G, N, lens = s["H"], s["P"], s["G"], s["N"], _lengths(s)
    dev, n, T, cu = "cuda", len(lens), sum(lens), s["cu"].long()
    per = (cu[1:] - cu[:-1] + Q - 1) // Q  # chunks of each document
    nc = int(sum(-(-m // Q) for m in lens))
    doc = torch.repeat_interleave(torch.arange(n, device=dev), per, output_size=nc)
    idx = torch.arange(nc, device=dev) - (torch.cumsum(per, 0) - per)[doc]  # chunk within its document
    tok = cu[doc][:, None] + idx[:, None] * Q + torch.arange(Q, device=dev)
    live = tok < cu[doc + 1][:, None]
    tok = torch.where(live, tok, 0)
    dt = torch.where(live[..., None], _softplus(s["dtr"].float() + s["dt_bias"])[tok], 0.0)  # [nc, Q, H]
    x, Bm, Cm = s["x"].float()[tok], s["B"].float()[tok], s["C"].float()[tok]  # [nc, Q, ...]
    la = torch.cumsum(dt * s["A"], 1).permute(0, 2, 1)  # [nc, H, Q]
    ends = la[..., -1]
    xd = (x * dt[..., None]).permute(0, 2, 1, 3)  # [nc, H, Q, P]
    Bh = Bm.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)
    Ch = Cm.permute(0, 2, 1, 3).repeat_interleave(H // G, 1)
    tri = torch.ones(Q, Q, device=dev, dtype=torch.bool).tril()
    L = torch.exp(torch.where(tri, la[..., :, None] - la[..., None, :], -math.inf))
    y = (L * (Ch @ Bh.transpose(-1, -2))) @ xd
    U = (Bh * torch.exp(ends[..., None] - la)[..., None]).transpose(-1, -2) @ xd  # each chunk's own state
    # The state at a chunk's start: earlier chunks of the same document, and the document's start state.
    upto = torch.cumsum(ends, 0)  # [nc, H]
    lo = upto - ends
    first = lo[torch.clamp((torch.cumsum(per, 0) - per)[doc], max=max(nc - 1, 0))]
    early = (doc[:, None] == doc[None, :]) & (idx[:, None] > idx[None, :])
    R = torch.exp(torch.where(early, lo.t()[:, :, None] - upto.t()[:, None, :], -math.inf))  # [H, nc, nc]
    U2 = U.permute(1, 0, 2, 3).reshape(H, nc, N * P)
    S0 = (R @ U2).view(H, nc, N, P).permute(1, 0, 2, 3)
    if s["s0"] is not None:
        S0 = S0 + s["s0"][doc] * torch.exp(lo - first)[..., None, None]
    y = y + (Ch @ S0) * torch.exp(la)[..., None]
    out = torch.empty(T, H, P, device=dev)
    out[tok[live]] = y.permute(0, 2, 1, 3)[live]
    ht = torch.zeros(n, H, N, P, device=dev) if s["s0"] is None else s["s0"].clone()
    final = idx == per[doc] - 1
    ht[doc[final]] = (S0 * torch.exp(ends)[..., None, None] + U)[final]
    return {"out": (out + s["Dskip"][:, None] * s["x"].float()).to(s["x"].dtype), "state": ht}


def _delta_step(s):
    slots, rep = s["slots"].long(), s["HV"] // s["Hqk"]
    q, k = s["q"].float(), s["k"].float()
    if s["l2"]:
        q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + EPS) for t in (q, k))
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    a = torch.exp(s["g"])
    S = s["state"][slots] * (a[..., None] if s["op"] == "kda" else a[..., None, None])
    d = s["beta"].float()[..., None] * (s["v"].float() - (S * k[..., None]).sum(2))
    S = S + k[..., None] * d[:, :, None, :]
    s["state"][slots] = S
    return {"out": (D ** -0.5 * (S * q[..., None]).sum(2)).to(torch.bfloat16), "state": s["state"]}


def _norm(s):
    t = s["x"].dtype
    x = s["x"].float()
    r1 = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r1 * s["w_post"].float() if s["post"] else x
    if s["gate"]:
        z = s["z"].float()
        sg = _sigmoid(z)
        act = z * sg if s["gate"] == "silu" else sg
        u = n * act
    else:
        u = n
    h = s["r"].float() + s["alpha"] * u if s["residual"] else u
    r2 = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    got = {}
    if s["residual"] or not s["pre"]:
        got["h"] = h.to(t)
    if s["pre"]:
        got["y"] = (h * r2 * s["w"].float()).to(t)
    if s["mode"] != "train":
        return got
    dh = s["dh"].float() if s["dh"] is not None else torch.zeros_like(h)
    if s["pre"]:
        dy, hn = s["dy"].float(), h * r2
        got["dweight"] = (dy * hn).sum((0, 1))
        dn = dy * s["w"].float()
        dh = dh + r2 * (dn - hn * (dn * hn).mean(-1, keepdim=True))
    if s["residual"]:
        got["dresidual"] = dh.to(t)
    du = s["alpha"] * dh
    if s["gate"]:
        got["dgate"] = (du * n * (_act_grad(z) if s["gate"] == "silu" else sg * (1 - sg))).to(t)
        du = du * act
    if s["post"]:
        xn = x * r1
        got["dpost_weight"] = (du * xn).sum((0, 1))
        dn = du * s["w_post"].float()
        du = r1 * (dn - xn * (dn * xn).mean(-1, keepdim=True))
    got["dx"] = du.to(t)
    return got


# ---------------------------------------------------------------------------
# Values in 64 bits, token by token and by the chain rule
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"sconv": _exact_conv, "ssm": _exact_ssm, "kda": _exact_delta, "gdn": _exact_delta, "norm": _exact_norm}[case["op"]](s)


def _exact_conv(s):
    w = s["weight"].double()
    b = s["b"].double() if s["b"] is not None else None
    K, C = s["W"] - 1, s["C"]
    f = (lambda z: z * torch.sigmoid(z)) if s["silu"] else (lambda z: z)
    if s["mode"] == "step":
        y, pool = torch.empty_like(s["x"], dtype=torch.float64), s["state"].double()
        for i, slot in enumerate(s["slots"].tolist()):
            seen = torch.cat([s["state"][slot].double(), s["x"][i:i + 1].double()])
            z = torch.einsum("jc,cj->c", seen, w)
            y[i] = f(z if b is None else z + b)
            pool[slot] = seen[1:]
        return {"out": y, "state": pool}
    train = s["mode"] == "train"
    outs, states, dxs, dw, db, at = [], [], [], torch.zeros_like(w), torch.zeros(C, dtype=torch.float64, device="cuda"), 0
    for i, m in enumerate(_lengths(s)):  # one document at a time
        x = s["x"][at:at + m].double()
        pre = s["s0"][i].double() if not train else x.new_zeros(K, C)
        seen = torch.cat([pre, x])
        z = x.new_zeros(m, C) if b is None else b.expand(m, C).clone()
        for j in range(K + 1):
            z += seen[j:j + m] * w[:, j]
        outs.append(f(z))
        states.append(seen[m:])
        if train:
            dz = s["dout"][at:at + m].double()
            if s["silu"]:
                e = torch.sigmoid(z)
                dz = dz * (e + z * e * (1 - e))
            dseen = torch.zeros_like(seen)
            for j in range(K + 1):
                dseen[j:j + m] += dz * w[:, j]
                dw[:, j] += (dz * seen[j:j + m]).sum(0)
            db += dz.sum(0)
            dxs.append(dseen[K:])
        at += m
    if not train:
        return {"out": torch.cat(outs), "state": torch.stack(states)}
    got = {"out": torch.cat(outs), "dx": torch.cat(dxs), "dweight": dw}
    if b is not None:
        got["dbias"] = db
    return got


def _exact_ssm(s):
    H, P, G, N = s["H"], s["P"], s["G"], s["N"]
    x, dt = s["x"].double(), torch.nn.functional.softplus(s["dtr"].double() + s["dt_bias"].double(), threshold=100.0)
    group = torch.arange(H, device="cuda") // (H // G)
    Bm, Cm = s["B"].double(), s["C"].double()
    decay = torch.exp(dt * s["A"].double())
    if s["mode"] == "step":
        pool, slots = s["state"].double(), s["slots"].long()
        S = torch.einsum("bh,bhnp->bhnp", decay, pool[slots])
        S = S + torch.einsum("bh,bhn,bhp->bhnp", dt, Bm[:, group], x)
        pool[slots] = S
        return {"out": torch.einsum("bhnp,bhn->bhp", S, Cm[:, group]) + s["Dskip"].double()[:, None] * x, "state": pool}
    lens = _lengths(s)
    n = len(lens)
    if max(lens, default=0) * n * H * N * P > 1 << 36:  # a walk of over about 20 seconds
        return None
    S = s["s0"].double() if s["s0"] is not None else torch.zeros(n, H, N, P, dtype=torch.float64, device="cuda")
    out = s["Dskip"].double()[:, None] * x
    starts = np.concatenate([[0], np.cumsum(lens)])[:-1]
    order = sorted(range(n), key=lambda i: -lens[i])  # longest first: those still running are the first ones
    S = S[torch.tensor(order, device="cuda")]
    first = torch.tensor([int(starts[i]) for i in order], device="cuda")
    dtx = dt[..., None] * x
    live = [0] * max(lens, default=0)
    for t in range(len(live)):
        live[t] = sum(lens[i] > t for i in order)
    for t, m in enumerate(live):
        at = first[:m] + t
        S[:m] *= decay[at][..., None, None]
        S[:m].view(m, G, H // G, N, P).add_(Bm[at][:, :, None, :, None] * dtx[at].view(m, G, H // G, 1, P))
        out[at] += torch.matmul(Cm[at][:, :, None, None, :], S[:m].view(m, G, H // G, N, P)).view(m, H, P)
    back = torch.empty_like(S)
    back[torch.tensor(order, device="cuda")] = S
    return {"out": out, "state": back}


def _exact_delta(s):
    q, k, v, beta, pool = (s[i].double() for i in ("q", "k", "v", "beta", "state"))
    y = torch.empty(s["batch"], s["HV"], D, dtype=torch.float64, device="cuda")
    if s["l2"]:
        q = q * (q.square().sum(-1, keepdim=True) + EPS).pow(-0.5)
        k = k * (k.square().sum(-1, keepdim=True) + EPS).pow(-0.5)
    for i, slot in enumerate(s["slots"].tolist()):
        qi = q[i].repeat_interleave(s["HV"] // s["Hqk"], 0)
        ki = k[i].repeat_interleave(s["HV"] // s["Hqk"], 0)
        a = torch.exp(s["g"][i].double())
        S = pool[slot] * (a[:, :, None] if s["op"] == "kda" else a[:, None, None])
        # (I - beta k k^T) S + beta k v^T
        S = S + beta[i][:, None, None] * torch.einsum("hc,hv->hcv", ki, v[i] - torch.einsum("hc,hcv->hv", ki, S))
        y[i] = D ** -0.5 * torch.einsum("hc,hcv->hv", qi, S)
        pool[slot] = S
    return {"out": y, "state": pool}


def _exact_norm(s):
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "z", "r", "w_post", "w") if s[k] is not None}
    with torch.enable_grad():
        u = leaf["x"]
        if s["post"]:
            u = u / torch.sqrt(u.square().mean(-1, keepdim=True) + EPS) * leaf["w_post"]
        if s["gate"]:
            u = u * torch.sigmoid(leaf["z"]) * (leaf["z"] if s["gate"] == "silu" else 1)
        h = leaf["r"] + s["alpha"] * u if s["residual"] else u
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * leaf["w"] if s["pre"] else None
        got = {}
        if s["residual"] or not s["pre"]:
            got["h"] = h.detach()
        if y is not None:
            got["y"] = y.detach()
        if s["mode"] == "train":
            total = 0
            if s["dh"] is not None:
                total = total + (h * s["dh"].double()).sum()
            if s["dy"] is not None:
                total = total + (y * s["dy"].double()).sum()
            names = {"x": "dx", "z": "dgate", "r": "dresidual", "w_post": "dpost_weight", "w": "dweight"}
            grads = torch.autograd.grad(total, list(leaf.values()))
            got.update({names[k]: v for k, v in zip(leaf, grads)})
    return got


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(c, work(c))
