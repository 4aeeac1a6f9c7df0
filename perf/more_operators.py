"""The softmax attention layer of a hybrid stack, as measured: cases, inputs, plain forms and 64-bit values.

Three families, each in the forms a program runs them in:

* lnorm: the scaled residual and the layer norm in front of a block (fwd, train);
* rope: rotary positions of q and k (fwd, train: the heads' rotation and their gradients' back);
* attn: attention over packed documents (fwd: prompts, prompts after a cache, single tokens; train: forward and
  backward).

A case is a dict of plain values; `lengths` lists the documents' tokens, `keys` their keys where they are not the
same.  `own` false computes the plain forms (elementary torch operations in 32 bits, angles in 64, rounded once at
the end), true calls the library.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
# Cached keys of 64 sequences being decoded, between one and some thousands.
CACHED = ",".join(str(1 + (i * 2654435761) % 8192) for i in range(64))


def listed():
    return [
        # One token of one sequence in front of a block: latency alone.
        {"name": "lnorm_b1", "op": "lnorm", "mode": "fwd", "rows": 1, "heads": 1, "D": 2048, "dtype": "bf16",
         "residual": True, "bias": True},
        # Training on a ragged pack of tokens: residual, norm, and the gradients of both and of weight and bias.
        {"name": "lnorm_train", "op": "lnorm", "mode": "train", "rows": 8191, "heads": 1, "D": 2048, "dtype": "bf16",
         "residual": True, "bias": True},
        # Training through a norm of each query head.
        {"name": "lnorm_train_heads", "op": "lnorm", "mode": "train", "rows": 32768, "heads": 16, "D": 128,
         "dtype": "bf16", "residual": False, "bias": False},
        # One token of one sequence, far into its text: latency alone.
        {"name": "rope_step_b1", "op": "rope", "mode": "fwd", "lengths": "1", "start": 1 << 20, "H": 16, "Hk": 4,
         "D": 128, "R": 128, "interleaved": False, "scaling": 1.0, "dtype": "bf16"},
        # Ragged prompts that go on behind cached tokens: half of each head, pairs side by side, a stretched context.
        {"name": "rope_prompt_ragged", "op": "rope", "mode": "fwd", "lengths": "1,129,0,2047,63,1000,3,858",
         "start": 5000, "H": 16, "Hk": 16, "D": 128, "R": 64, "interleaved": True, "scaling": 8.0, "dtype": "f16"},
        # Training on a long document with grouped heads.
        {"name": "rope_train_32k", "op": "rope", "mode": "train", "lengths": "32768", "start": 0, "H": 32, "Hk": 8,
         "D": 128, "R": 128, "interleaved": False, "scaling": 1.0, "dtype": "bf16"},
        # Short prompts of odd lengths, one of them empty.
        {"name": "attn_prompt_ragged", "op": "attn", "mode": "fwd", "lengths": "1,63,64,0,65,129,300", "keys": "",
         "H": 16, "Hk": 16, "D": 128, "causal": True, "window": 0},
        # One token of each of 64 sequences against its keys.
        {"name": "attn_step_b64", "op": "attn", "mode": "fwd", "lengths": ",".join(["1"] * 64), "keys": CACHED,
         "H": 32, "Hk": 8, "D": 128, "causal": True, "window": 0},
        # One long prompt with grouped heads.
        {"name": "attn_prompt_32k", "op": "attn", "mode": "fwd", "lengths": "32768", "keys": "", "H": 16, "Hk": 4,
         "D": 128, "causal": True, "window": 0},
        # Training on a few short documents with few heads: latency.
        {"name": "attn_train_short", "op": "attn", "mode": "train", "lengths": "300,17,1,511,128", "keys": "", "H": 4,
         "Hk": 4, "D": 64, "causal": True, "window": 0},
        # Training on one document with grouped heads.
        {"name": "attn_train_8k", "op": "attn", "mode": "train", "lengths": "8192", "keys": "", "H": 16, "Hk": 4,
         "D": 128, "causal": True, "window": 0},
        # Training on ragged documents through a layer that sees the last 1024 tokens.
        {"name": "attn_train_window", "op": "attn", "mode": "train", "lengths": "5000,1,11383,777", "keys": "", "H": 16,
         "Hk": 16, "D": 64, "causal": True, "window": 1024},
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
    op = rng.choice(["lnorm", "rope", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "lnorm":
        heads = rng.choice([1, 1, 4, 16, 48])
        width = _log_int(rng, 16, 8192) if heads == 1 else rng.choice([64, 128, 256])
        if heads == 1 and rng.random() < 0.6:
            width = -(-width // 8) * 8
        return {"op": op, "mode": rng.choice(["fwd", "train"]), "rows": _log_int(rng, 1, min(32768, (1 << 27) // (BYTES[dtype] * heads * width))),
                "heads": heads, "D": width, "dtype": dtype, "residual": heads == 1 and rng.random() < 0.6,
                "bias": rng.random() < 0.5}
    if op == "rope":
        Hk, G = rng.choice([(1, 1), (1, 8), (4, 4), (8, 4), (16, 1), (3, 5)])
        D = rng.choice([32, 64, 80, 96, 128, 128, 256])
        return {"op": op, "mode": rng.choice(["fwd", "train"]), "lengths": _cut(rng, _log_int(rng, 1, 65536 * 128 // (BYTES[dtype] * max(128, D)))),
                "start": rng.choice([0, 0, _log_int(rng, 1, 1 << 22)]), "H": Hk * G, "Hk": Hk, "D": D,
                "R": rng.choice([D, D, D // 2, D // 4]), "interleaved": rng.random() < 0.5,
                "scaling": rng.choice([1.0, 1.0, 4.0, 32.0]), "dtype": dtype}
    Hk, G = rng.choice([(1, 1), (2, 1), (16, 1), (4, 4), (2, 8), (1, 8), (8, 3), (3, 5)])
    kind = rng.choice(["fwd", "train", "train", "after", "step"])
    case = {"op": op, "mode": "train" if kind == "train" else "fwd", "H": Hk * G, "Hk": Hk,
            "D": rng.choice([64, 128, 128, 128, 32, 80, 96]), "causal": True, "window": 0}
    if kind == "step":
        n = _log_int(rng, 1, 64)
        case.update(lengths=",".join(["1"] * n), keys=",".join(str(_log_int(rng, 1, min(65536, (1 << 17) // n))) for _ in range(n)))
    elif kind == "after":  # most documents see more keys than they have tokens, some fewer: their first tokens see none
        lens = [int(n) for n in _cut(rng, _log_int(rng, 1, 4096)).split(",")]
        case.update(lengths=",".join(map(str, lens)), keys=",".join(str(max(0, n + rng.choice([-5, 0, 7, 1000, 4096]))) for n in lens))
    else:
        # at most the work of the long prompt with 16 heads, forward and backward
        most = 24576 if kind == "fwd" else 11264
        # (a token alone has no gradient of q and k but rounding errors: at least one document of two)
        case.update(lengths=_cut(rng, _log_int(rng, 1 if kind == "fwd" else 16, most)), keys="", causal=rng.random() < 0.8)
    if case["causal"]:
        case["window"] = rng.choice([0, 0, 0, 128, 1000])
    return case


def _ints(text):
    return [int(n) for n in text.split(",")]


def _lens(case):
    """Tokens and keys of each document."""
    q = _ints(case["lengths"])
    return q, _ints(case["keys"]) if case["keys"] else q


def _pairs(case):
    """How many (query, key) pairs the mask leaves."""
    total = 0
    for lq, lk in zip(*_lens(case)):
        if not case["causal"]:
            total += lq * lk
            continue
        last = np.arange(lk - lq + 1, lk + 1)  # keys that a query sees without a window
        seen = np.clip(last, 0, case["window"] or None)
        total += int(seen.sum())
    return total


def work(case):
    op, train = case["op"], case["mode"] == "train"
    if op == "lnorm":
        n, e, res = case["rows"] * case["heads"] * case["D"], BYTES[case["dtype"]], case["residual"]
        moved = 2 + 2 * res  # x, y; with the residual its input and its sum
        if train:
            moved += 3 + 3 * res  # x, dy, dx; the residual, its sum's gradient, its own gradient
        return {"bytes": n * e * moved + 4.0 * case["D"], "flops": n * (8.0 if not train else 24.0)}
    if op == "rope":
        n = sum(_ints(case["lengths"])) * (case["H"] + case["Hk"]) * case["D"]
        return {"bytes": n * BYTES[case["dtype"]] * (4 if train else 2), "flops": n * (6.0 if train else 3.0)}
    H, Hk, D = case["H"], case["Hk"], case["D"]
    tq, tk = (sum(x) for x in _lens(case))
    moved = 2 * tq * H * D + 2 * tk * Hk * D  # q, out; k, v
    if train:  # q, out, dout, dq; k, v, dk, dv
        moved += 4 * tq * H * D + 4 * tk * Hk * D
    # two products of the scores' size forward, five backward
    return {"bytes": 2 * moved + 4 * tq * H, "flops": (14.0 if train else 4.0) * _pairs(case) * H * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pack(lens):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return cu, torch.from_numpy(cu).cuda()


def _frequencies(R, factor, base=10000.0, context=4096, slow=1.0, fast=32.0):
    """Radians a token of the R / 2 pairs; a context stretched by `factor` slows the pairs that turn less than
    `fast` times within the original one (those below `slow` wholly)."""
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if factor != 1.0:
        keep = np.clip((f * context / (2 * math.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * (keep + (1 - keep) / factor)
    return torch.from_numpy(f.astype(np.float32)).cuda()


def prepare(case, seed):
    g, op, train = _gen(seed), case["op"], case["mode"] == "train"
    s = dict(case)
    if op == "lnorm":
        t, shape, D = DTYPES[case["dtype"]], (case["rows"], case["heads"], case["D"]), case["D"]
        s["x"] = (_randn(g, *shape) + 0.5 * _randn(g, shape[0], shape[1], 1)).to(t)
        s["r"] = (2 * _randn(g, *shape)).to(t) if case["residual"] else None
        s["w"] = (1 + 0.1 * _randn(g, D)).to(t)
        s["b"] = (0.1 * _randn(g, D)).to(t) if case["bias"] else None
        s["alpha"] = 0.5 if case["residual"] else 1.0
        if train:
            s["dh"] = _randn(g, *shape).to(t) if case["residual"] else None
            s["dy"] = _randn(g, *shape).to(t)
        return s
    H, Hk, D = case["H"], case["Hk"], case["D"]
    if op == "rope":
        t, lens = DTYPES[case["dtype"]], _ints(case["lengths"])
        T = sum(lens)
        # q and k are slices of one projection
        for names in (("q", "k"), ("dq", "dk")) if train else (("q", "k"),):
            qkv = _randn(g, T, (H + 2 * Hk) * D).to(t)
            s[names[0]] = qkv[:, : H * D].unflatten(1, (H, D))
            s[names[1]] = qkv[:, H * D: (H + Hk) * D].unflatten(1, (Hk, D))
        at = np.concatenate([np.arange(n) for n in lens]) + case["start"]
        s["positions"] = torch.from_numpy(at.astype(np.int32)).cuda()
        s["freqs"] = _frequencies(case["R"], case["scaling"])
        s["amp"] = 0.1 * math.log(case["scaling"]) + 1.0
        return s
    (lq, lk), bf = _lens(case), torch.bfloat16
    s["cu_host"], s["cu"] = _pack(lq)
    s["cuk_host"], s["cuk"] = _pack(lk) if case["keys"] else (None, None)
    if case["keys"]:  # the keys and values lie in a cache of their own
        s["q"] = _randn(g, sum(lq), H, D).to(bf)
        s["k"], s["v"] = (_randn(g, sum(lk), Hk, D).to(bf) for _ in range(2))
    else:  # q, k and v are slices of one projection
        qkv = _randn(g, sum(lq), (H + 2 * Hk) * D).to(bf)
        s["q"] = qkv[:, : H * D].unflatten(1, (H, D))
        s["k"] = qkv[:, H * D: (H + Hk) * D].unflatten(1, (Hk, D))
        s["v"] = qkv[:, (H + Hk) * D:].unflatten(1, (Hk, D))
    if train:
        s["dout"] = _randn(g, sum(lq), H, D).to(bf)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    if own:
        return _run_own(s)
    return {"lnorm": _lnorm, "rope": _rope, "attn": _attn}[s["op"]](s)


def _run_own(s):
    import gated_delta_rule_varlen_gb300 as gdr

    op, train = s["op"], s["mode"] == "train"
    if op == "lnorm":
        args = dict(residual=s["r"], res_scale=s["alpha"], eps=EPS)
        h, y = gdr.lnorm_fwd(s["x"], s["w"], s["b"], **args)
        got = {"h": h, "y": y}
        if train:
            got.update(gdr.lnorm_bwd(s["x"], s["w"], s["b"], dh=s["dh"], dy=s["dy"], **args))
        return {k: v for k, v in got.items() if v is not None}
    if op == "rope":
        args = dict(positions=s["positions"], interleaved=s["interleaved"], amplitude=s["amp"])
        q, k = gdr.rope_fwd(s["q"], s["k"], s["freqs"], **args)
        got = {"q": q, "k": k}
        if train:
            got["dq"], got["dk"] = gdr.rope_bwd(s["dq"], s["dk"], s["freqs"], **args)
        return got
    pack, args = (s["cu"], s["cu_host"]), dict(causal=s["causal"], window=s["window"], cu_keys=s["cuk"], cu_keys_host=s["cuk_host"])
    out, lse = gdr.attn_fwd(s["q"], s["k"], s["v"], *pack, **args)
    got = {"out": out, "lse": lse}
    if train:
        got.update(gdr.attn_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], *pack, **args))
    return got


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _lnorm(s):
    t = s["x"].dtype
    h = s["x"].float()
    if s["residual"]:
        h = s["r"].float() + s["alpha"] * h
    d = h - h.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n, w = d * r, s["w"].float()
    y = n * w + s["b"].float() if s["bias"] else n * w
    got = {"y": y.to(t)}
    if s["residual"]:
        got["h"] = h.to(t)
    if s["mode"] != "train":
        return got
    dy = s["dy"].float()
    got["dweight"] = (dy * n).sum((0, 1))
    if s["bias"]:
        got["dbias"] = dy.sum((0, 1))
    dn = dy * w
    dh = r * (dn - dn.mean(-1, keepdim=True) - n * (dn * n).mean(-1, keepdim=True))
    if s["residual"]:
        dh = dh + s["dh"].float()
        got["dresidual"] = dh.to(t)
        dh = s["alpha"] * dh
    got["dx"] = dh.to(t)
    return got


def _turn(x, cos, sin, R, interleaved):
    f = x.float()
    a, b = (f[..., 0:R:2], f[..., 1:R:2]) if interleaved else (f[..., : R // 2], f[..., R // 2: R])
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, f[..., R:]], -1).to(x.dtype)


def _rope(s):
    angle = s["positions"].double()[:, None] * s["freqs"].double()  # far positions lose their angle in 32 bits
    cos, sin = ((s["amp"] * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))
    got = {n: _turn(s[n], cos, sin, s["R"], s["interleaved"]) for n in ("q", "k")}
    if s["mode"] == "train":
        got.update({n: _turn(s[n], cos, -sin, s["R"], s["interleaved"]) for n in ("dq", "dk")})
    return got


def _hidden(s, lq, lk, i0, i1, j0, j1):
    """Which of the keys [j0, j1) the queries [i0, i1) do not see; None: none."""
    if not s["causal"]:
        return None
    i = torch.arange(i0, i1, device="cuda")[:, None] + (lk - lq)
    j = torch.arange(j0, j1, device="cuda")[None, :]
    return (j > i) | (j <= i - s["window"]) if s["window"] else j > i


def _softmax(x, hidden):
    """exp(x - lse) and lse over the last dimension; a row that sees nothing: zeros and -inf."""
    if hidden is not None:
        x = torch.where(hidden, -math.inf, x)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else x.new_full((*x.shape[:-1], 1), -math.inf)
    p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0), (top + torch.log(total)).squeeze(-1)


def _attn(s):
    lq, lk = _lens(s)
    if s["mode"] == "fwd" and max(lq) == 1:
        return _attn_step(s)
    H, Hk, D, train = s["H"], s["Hk"], s["D"], s["mode"] == "train"
    G, c, T = H // Hk, D ** -0.5, sum(lq)
    got = {"out": torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), "lse": torch.empty(H, T, device="cuda")}
    if train:
        got["dq"] = torch.empty_like(got["out"])
        got["dk"], got["dv"] = (torch.zeros(sum(lk), Hk, D, device="cuda") for _ in range(2))
    a = b = 0
    for n, m in zip(lq, lk):
        k, v = (s[x][b:b + m].float().permute(1, 0, 2)[:, None] for x in ("k", "v"))  # [Hk, 1, m, D]
        step = max(1, (1 << 28) // max(1, H * m))
        for i in range(0, n, step):
            e = min(n, i + step)
            top = max(0, min(m, e + m - n)) if s["causal"] else m  # keys behind the block's last query
            low = max(0, min(top, i + m - n - s["window"] + 1)) if s["window"] else 0
            kk, vv = k[:, :, low:top], v[:, :, low:top]
            q = s["q"][a + i:a + e].float().view(e - i, Hk, G, D).permute(1, 2, 0, 3)  # [Hk, G, rows, D]
            p, lse = _softmax(c * (q @ kk.transpose(-1, -2)), _hidden(s, n, m, i, e, low, top))
            o = p @ vv
            got["out"][a + i:a + e] = o.permute(2, 0, 1, 3).reshape(e - i, H, D).to(torch.bfloat16)
            got["lse"][:, a + i:a + e] = lse.reshape(H, e - i)
            if train:
                do = s["dout"][a + i:a + e].float().view(e - i, Hk, G, D).permute(1, 2, 0, 3)
                ds = p * (do @ vv.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
                got["dq"][a + i:a + e] = (c * (ds @ kk)).permute(2, 0, 1, 3).reshape(e - i, H, D).to(torch.bfloat16)
                got["dv"][b + low:b + top] += (p.transpose(-1, -2) @ do).sum(1).transpose(0, 1)
                got["dk"][b + low:b + top] += c * (ds.transpose(-1, -2) @ q).sum(1).transpose(0, 1)
        a, b = a + n, b + m
    if train:
        got["dk"], got["dv"] = got["dk"].to(torch.bfloat16), got["dv"].to(torch.bfloat16)
    return got


def _attn_step(s):
    """Tokens of one a document at most: the keys of all documents side by side, padded."""
    lq, lk = _lens(s)
    H, Hk, D, dev = s["H"], s["Hk"], s["D"], "cuda"
    G = H // Hk
    cuk = (s["cuk"] if s["cuk"] is not None else s["cu"]).long()
    doc = torch.repeat_interleave(torch.arange(len(lq), device=dev), (s["cu"][1:] - s["cu"][:-1]).long(), output_size=sum(lq))
    n = (cuk[1:] - cuk[:-1])[doc]
    at = torch.arange(max(lk), device=dev)
    gone = at >= n[:, None]
    if s["window"]:
        gone = gone | (at <= n[:, None] - 1 - s["window"])
    rows = torch.where(at < n[:, None], cuk[:-1][doc][:, None] + at, 0)
    q = s["q"].float().view(-1, Hk, G, D)
    k, v = (s[x][rows].float().permute(0, 2, 1, 3) for x in ("k", "v"))  # [batch, Hk, keys, D]
    p, lse = _softmax(D ** -0.5 * (q @ k.transpose(-1, -2)), gone[:, None, None, :])
    v = torch.where(gone[:, None, :, None], 0.0, v)
    return {"out": (p @ v).reshape(-1, H, D).to(torch.bfloat16), "lse": lse.reshape(-1, H).t().contiguous()}


# ---------------------------------------------------------------------------
# Values in 64 bits, by torch's own norm, complex rotations and one head at a time
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] * (1 if case["causal"] and not case["window"] else 4) > 6e12:
        return None  # over about 20 seconds
    s = prepare(case, seed)
    return {"lnorm": _exact_lnorm, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](s)


def _exact_lnorm(s):
    leaf = {k: s[k].double().requires_grad_() for k in ("x", "r", "w", "b") if s[k] is not None}
    with torch.enable_grad():
        h = leaf["r"] + s["alpha"] * leaf["x"] if s["residual"] else leaf["x"]
        var, mean = torch.var_mean(h, -1, correction=0, keepdim=True)
        y = (h - mean) / torch.sqrt(var + EPS) * leaf["w"] + leaf.get("b", 0.0)
        got = {"y": y.detach()}
        if s["residual"]:
            got["h"] = h.detach()
        if s["mode"] == "train":
            total = (y * s["dy"].double()).sum()
            if s["residual"]:
                total = total + (h * s["dh"].double()).sum()
            names = {"x": "dx", "r": "dresidual", "w": "dweight", "b": "dbias"}
            got.update({names[k]: v for k, v in zip(leaf, torch.autograd.grad(total, list(leaf.values())))})
    return got


def _exact_rope(s):
    R, got = s["R"], {}
    angle = torch.outer(s["positions"].double(), s["freqs"].double())
    for n in ("q", "k", "dq", "dk"):
        if n not in s:
            continue
        x = s[n].double()
        z = x[..., :R].unflatten(-1, (R // 2, 2)) if s["interleaved"] else x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
        turn = torch.polar(torch.full_like(angle, s["amp"]), -angle if n[0] == "d" else angle)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn[:, None, :])
        z = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
        got[n] = torch.cat([z, x[..., R:]], -1)
    return got


def _exact_attn(s):
    lq, lk = _lens(s)
    H, Hk, D, train, f64 = s["H"], s["Hk"], s["D"], s["mode"] == "train", torch.float64
    G, T, Tk = H // Hk, sum(lq), sum(lk)
    got = {"out": torch.zeros(T, H, D, dtype=f64, device="cuda"), "lse": torch.full((H, T), -math.inf, dtype=f64, device="cuda")}
    if train:
        got.update(dq=torch.zeros(T, H, D, dtype=f64, device="cuda"), dk=torch.zeros(Tk, Hk, D, dtype=f64, device="cuda"),
                   dv=torch.zeros(Tk, Hk, D, dtype=f64, device="cuda"))
    a = b = 0
    for n, m in zip(lq, lk):
        if m and n:
            for h in range(H):
                K, V = s["k"][b:b + m, h // G].double(), s["v"][b:b + m, h // G].double()
                for i in range(0, n, 4096):
                    e = min(n, i + 4096)
                    # the keys that any of these queries sees
                    last = min(m, m - n + e) if s["causal"] else m
                    first = max(0, m - n + i + 1 - s["window"]) if s["window"] else 0
                    if last <= first:
                        continue
                    Q, at = s["q"][a + i:a + e, h].double(), slice(first, last)
                    S = torch.addmm(torch.zeros((), dtype=f64, device="cuda"), Q, K[at].t(), beta=0, alpha=1 / math.sqrt(D))
                    if s["causal"]:
                        gap = (torch.arange(i, e, device="cuda") + m - n)[:, None] - torch.arange(first, last, device="cuda")
                        seen = (gap >= 0) & (gap < s["window"]) if s["window"] else gap >= 0
                        S.masked_fill_(~seen, -math.inf)
                    lse = torch.logsumexp(S, -1)
                    got["lse"][h, a + i:a + e] = lse
                    P = torch.softmax(S, -1)
                    P[lse == -math.inf] = 0
                    got["out"][a + i:a + e, h] = P @ V[at]
                    if train:
                        dO = s["dout"][a + i:a + e, h].double()
                        got["dv"][b + first:b + last, h // G] += P.t() @ dO
                        dP = dO @ V[at].t()
                        dS = P * (dP - (P * dP).sum(-1, keepdim=True)) / math.sqrt(D)
                        got["dq"][a + i:a + e, h] = dS @ K[at]
                        got["dk"][b + first:b + last, h // G] += dS.t() @ Q
        a, b = a + n, b + m
    return got


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(c, work(c))
