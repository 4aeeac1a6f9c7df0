"""Three token mixers built from the library's operators, in training, on prompts
and token by token:

* a grouped GDN layer: norm -> projections -> short convolution (+ SiLU) on q, k
  and v -> gated delta rule (q, k normalized in the kernels) -> per-head norm and
  gate -> output projection;
* a scan layer: norm -> projections -> short convolution on x, B and C -> selective
  state space scan -> norm and gate -> output projection;
* a softmax attention layer: layer norm -> projections -> rotary positions on q and k ->
  attention over the document's tokens and the cached keys before them -> output projection;

between the first two the residual, its scale and the next norm in one pass.  Run as a
program it checks that serving continues a prompt (the same text as one prompt,
and as a prompt followed by single tokens from the cached states) and that a
training step's gradients agree with differences, and prints what each form took:

    python examples/hybrid_layers.py
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_varlen_gb300 as gdr  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
W = 4  # taps of the convolutions


def randn(g, *shape, scale=1.0, dtype=BF16):
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


class GdnMixer:
    """Grouped GDN: Hqk query/key heads and HV value heads of 128."""

    def __init__(self, g, width, Hqk, HV):
        self.width, self.Hqk, self.HV = width, Hqk, HV
        self.channels = (2 * Hqk + HV) * 128
        cols = self.channels + HV * 128 + 2 * HV  # q k v | output gate | decay, beta
        self.w_in = randn(g, width, cols, scale=width ** -0.5)
        self.conv = randn(g, self.channels, W, scale=0.5)
        self.out_norm = torch.ones(128, device="cuda", dtype=BF16)
        self.w_out = randn(g, HV * 128, width, scale=(HV * 128) ** -0.5)

    def _project(self, x):
        p = x @ self.w_in
        qkv, z, ab = p[:, :self.channels], p[:, self.channels:-2 * self.HV], p[:, -2 * self.HV:].float()
        g = -torch.nn.functional.softplus(ab[:, :self.HV] - 2)
        return qkv, z.unflatten(1, (self.HV, 128)), g.contiguous(), torch.sigmoid(ab[:, self.HV:]).contiguous()

    def _split(self, y):
        a, b = self.Hqk * 128, 2 * self.Hqk * 128
        return (y[:, :a].unflatten(1, (self.Hqk, 128)).contiguous(), y[:, a:b].unflatten(1, (self.Hqk, 128)).contiguous(),
                y[:, b:].unflatten(1, (self.HV, 128)).contiguous())

    def prompt(self, x, cu, cu_host, state=None):
        conv0, h0 = state if state is not None else (None, None)
        qkv, z, g, beta = self._project(x)
        y, conv = gdr.sconv_fwd(qkv, self.conv, None, cu, cu_host, s0=conv0)
        o, h, _ = gdr.gdn_fwd(*self._split(y), g, beta, cu, cu_host, 128 ** -0.5, h0=h0, save_for_bwd=False, qk_l2norm=True)
        o, _ = gdr.norm_fwd(o, post_weight=self.out_norm, gate=z)
        return o.flatten(1) @ self.w_out, (conv, h)

    def step(self, x, state, slots=None):
        conv, h = state
        qkv, z, g, beta = self._project(x)
        y = gdr.sconv_step(qkv, self.conv, None, conv, slots=slots)
        o = gdr.gdn_step(*self._split(y), g, beta, h, 128 ** -0.5, slots=slots, qk_l2norm=True)
        o, _ = gdr.norm_fwd(o, post_weight=self.out_norm, gate=z)
        return o.flatten(1) @ self.w_out

    def train(self, x, cu, cu_host, dout):
        """Forward, and the gradients of sum(out * dout) with respect to the convolution and the output norm."""
        qkv, z, g, beta = self._project(x)
        y, _ = gdr.sconv_fwd(qkv, self.conv, None, cu, cu_host, want_st=False)
        q, k, v = self._split(y)
        o, _, saved = gdr.gdn_fwd(q, k, v, g, beta, cu, cu_host, 128 ** -0.5, want_ht=False, qk_l2norm=True)
        n, _ = gdr.norm_fwd(o, post_weight=self.out_norm, gate=z)
        out = n.flatten(1) @ self.w_out
        dn = (dout @ self.w_out.t()).unflatten(1, (self.HV, 128))
        gn = gdr.norm_bwd(o, post_weight=self.out_norm, gate=z, dh=dn)
        gg = gdr.gdn_bwd(q, k, v, g, beta, cu, cu_host, 128 ** -0.5, gn["dx"], saved, qk_l2norm=True)
        dy = torch.cat([gg["dq"].flatten(1), gg["dk"].flatten(1), gg["dv"].flatten(1)], 1)
        gc = gdr.sconv_bwd(qkv, self.conv, None, cu, cu_host, dy)
        return out, {"conv": gc["dweight"], "out_norm": gn["dpost_weight"]}


class ScanMixer:
    """Selective scan: H heads of P, state size N, G groups of B and C."""

    def __init__(self, g, width, H, P, G, N):
        self.H, self.P, self.G, self.N = H, P, G, N
        self.inner, self.channels = H * P, H * P + 2 * G * N
        self.w_in = randn(g, width, self.inner + self.channels + H, scale=width ** -0.5)
        self.conv, self.conv_bias = randn(g, self.channels, W, scale=0.5), randn(g, self.channels, scale=0.1)
        self.A = -(1 + 15 * torch.rand(H, generator=g, device="cuda"))
        self.dt_bias = -4 + 2 * torch.rand(H, generator=g, device="cuda")
        self.D = torch.ones(H, device="cuda")
        self.out_norm = torch.ones(self.inner, device="cuda", dtype=BF16)
        self.w_out = randn(g, self.inner, width, scale=self.inner ** -0.5)

    def _project(self, x):
        p = x @ self.w_in
        return p[:, :self.inner], p[:, self.inner:self.inner + self.channels], p[:, self.inner + self.channels:]

    def _split(self, y):  # slices of the convolution's rows, as they are
        a, b = self.inner, self.inner + self.G * self.N
        return y[:, :a].unflatten(1, (self.H, self.P)), y[:, a:b].unflatten(1, (self.G, self.N)), y[:, b:].unflatten(1, (self.G, self.N))

    def prompt(self, x, cu, cu_host, state=None):
        conv0, h0 = state if state is not None else (None, None)
        z, xbc, dt = self._project(x)
        y, conv = gdr.sconv_fwd(xbc, self.conv, self.conv_bias, cu, cu_host, s0=conv0)
        xs, B, C = self._split(y)
        o, h = gdr.ssm_fwd(xs, dt, self.A, B, C, cu, cu_host, D=self.D, dt_bias=self.dt_bias, h0=h0)
        o, _ = gdr.norm_fwd(o.flatten(1), post_weight=self.out_norm, gate=z)
        return o @ self.w_out, (conv, h)

    def step(self, x, state, slots=None):
        conv, h = state
        z, xbc, dt = self._project(x)
        xs, B, C = self._split(gdr.sconv_step(xbc, self.conv, self.conv_bias, conv, slots=slots))
        o = gdr.ssm_step(xs, dt, self.A, B, C, h, D=self.D, dt_bias=self.dt_bias, slots=slots)
        o, _ = gdr.norm_fwd(o.flatten(1), post_weight=self.out_norm, gate=z)
        return o @ self.w_out


class AttentionMixer:
    """Softmax attention of H query heads over HK key heads of D; the state is each
    document's keys and values so far, packed as `lengths` says."""

    def __init__(self, g, width, H, HK, D):
        self.H, self.HK, self.D = H, HK, D
        self.norm_weight, self.norm_bias = torch.ones(width, device="cuda"), randn(g, width, scale=0.1, dtype=F32)
        self.w_in = randn(g, width, (H + 2 * HK) * D, scale=width ** -0.5)
        self.w_out = randn(g, H * D, width, scale=(H * D) ** -0.5)
        self.freqs = gdr.rope_frequencies(D, scaling="parts", factor=4.0)

    def _project(self, x, positions):
        _, y = gdr.lnorm_fwd(x, self.norm_weight, self.norm_bias)
        a, b = self.H * self.D, (self.H + self.HK) * self.D
        p = y @ self.w_in
        q, k, v = (s.unflatten(1, (-1, self.D)) for s in (p[:, :a], p[:, a:b], p[:, b:]))  # slices, as they are
        return *gdr.rope_fwd(q, k, self.freqs, positions=positions), v

    def prompt(self, x, cu, cu_host, state=None):
        new = [b - a for a, b in zip(cu_host, cu_host[1:])]
        old, keys, values = state if state is not None else ([0] * len(new), None, None)
        positions = torch.cat([torch.arange(a, a + n) for a, n in zip(old, new)]).to("cuda", torch.int32)
        q, k, v = self._project(x, positions)
        lengths, args = [a + n for a, n in zip(old, new)], {}
        if state is not None:
            k, v = (torch.cat([t for pair in zip(c.split(old), n.split(new)) for t in pair]) for c, n in ((keys, k), (values, v)))
            args = dict(zip(("cu_keys", "cu_keys_host"), pack(lengths)))
        o, _ = gdr.attn_fwd(q, k, v, cu, cu_host, **args)
        return o.flatten(1) @ self.w_out, (lengths, k, v)

    def train(self, x, cu, cu_host, dout):
        """Forward, and the gradients of sum(out * dout) with respect to the norm's weight and bias."""
        q, k, v = self._project(x, torch.cat([torch.arange(b - a) for a, b in zip(cu_host, cu_host[1:])]).to("cuda", torch.int32))
        o, lse = gdr.attn_fwd(q, k, v, cu, cu_host)
        out = o.flatten(1) @ self.w_out
        ga = gdr.attn_bwd(q, k, v, o, lse, (dout @ self.w_out.t()).unflatten(1, (self.H, self.D)), cu, cu_host)
        dq, dk = gdr.rope_bwd(ga["dq"], ga["dk"], self.freqs, cu_seqlens=cu)
        dy = torch.cat([dq.flatten(1), dk.flatten(1), ga["dv"].flatten(1)], 1) @ self.w_in.t()
        gn = gdr.lnorm_bwd(x, self.norm_weight, self.norm_bias, dy=dy)
        return out, {"norm_weight": gn["dweight"], "norm_bias": gn["dbias"]}


class Model:
    def __init__(self, seed, width=512, Hqk=2, HV=4, H=8, P=64, G=1, N=128, depth=2):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.mixers = [m for _ in range(depth) for m in (GdnMixer(g, width, Hqk, HV), ScanMixer(g, width, H, P, G, N))]
        self.norms = [torch.ones(width, device="cuda", dtype=BF16) for _ in range(len(self.mixers) + 1)]
        self.scale = (2 * depth) ** -0.5  # of each block's output on the residual

    def _run(self, x, mix):
        h, y = x, gdr.norm_fwd(x, weight=self.norms[0])[1]
        for i, m in enumerate(self.mixers):
            # residual + scale * block, and the next block's norm, in one pass
            h, y = gdr.norm_fwd(mix(i, m, y), weight=self.norms[i + 1], residual=h, res_scale=self.scale)
        return y

    def prompt(self, x, cu, cu_host, states=None):
        kept = [None] * len(self.mixers)

        def mix(i, m, y):
            out, kept[i] = m.prompt(y, cu, cu_host, None if states is None else states[i])
            return out
        return self._run(x, mix), kept

    def step(self, x, states, slots=None):
        return self._run(x, lambda i, m, y: m.step(y, states[i], slots))


def pack(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device="cuda"), cu


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def serve(model, lengths, more, width=512, seed=1):
    """(relative difference of the last `more` tokens' outputs: one prompt against prompt + steps)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    texts = [randn(g, n + more, width) for n in lengths]
    whole, _ = model.prompt(torch.cat(texts), *pack([n + more for n in lengths]))
    want = [t[-more:] for t in whole.split([n + more for n in lengths])]
    _, states = model.prompt(torch.cat([t[:-more] for t in texts]), *pack(lengths))
    got = torch.stack([model.step(torch.stack([t[n + i] for t, n in zip(texts, lengths)]), states) for i in range(more)], 1)
    return rel(got, torch.stack(want))


def attend(mixer, lengths, more, width=512, seed=3):
    """The same of an attention layer alone: prompt, the keys it leaves, and single tokens after them."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    texts = [randn(g, n + more, width) for n in lengths]
    whole, _ = mixer.prompt(torch.cat(texts), *pack([n + more for n in lengths]))
    want = [t[-more:] for t in whole.split([n + more for n in lengths])]
    _, state = mixer.prompt(torch.cat([t[:-more] for t in texts]), *pack(lengths))
    got, each = [], pack([1] * len(lengths))
    for i in range(more):
        out, state = mixer.prompt(torch.stack([t[n + i] for t, n in zip(texts, lengths)]), *each, state)
        got.append(out)
    return rel(torch.stack(got, 1), torch.stack(want))


def train(m, names, lengths, width=512, seed=2):
    """(relative difference of the directional derivative by differences from the gradients', for each parameter)"""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = sum(lengths)
    x, dout, cu = randn(g, T, width), randn(g, T, width), pack(lengths)
    _, grads = m.train(x, *cu, dout)
    got = {}
    for name in names:
        p = getattr(m, name)
        v, eps = grads[name] / grads[name].norm(), 0.25 if name == "conv" else 0.5
        loss = []
        for sign in (1, -1):
            setattr(m, name, (p.float() + sign * eps * v).contiguous())  # FP32 parameters beside BF16 activations
            out, _ = m.train(x, *cu, dout)
            loss.append(float((out.double() * dout.double()).sum()))
        setattr(m, name, p)
        want = float((grads[name] * v).sum())
        got[name] = abs((loss[0] - loss[1]) / (2 * eps) - want) / abs(want)
    return got


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--lengths", default="300,65,1,128")
    ap.add_argument("--more", type=int, default=24)
    a = ap.parse_args(argv)
    lengths = [int(n) for n in a.lengths.split(",")]
    model = Model(0)
    serve(model, lengths, 2)  # warm-up
    d = serve(model, lengths, a.more)
    t = train(model.mixers[0], ("conv", "out_norm"), lengths)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    mixer = AttentionMixer(g, 512, 8, 2, 64)
    da = attend(mixer, lengths, a.more)
    t.update(train(mixer, ("norm_weight", "norm_bias"), lengths))
    gdr.gdr_check_device()
    print(f"serving: outputs of {a.more} single tokens after the prompts differ by {d:.2e} from one prompt of all, {da:.2e} of attention")
    print("training: gradients and differences apart by " + ", ".join(f"{k} {v:.2e}" for k, v in t.items()))
    gdr.gdr_profile_enable(True)
    serve(model, lengths, a.more)
    train(model.mixers[0], ("conv", "out_norm"), lengths)
    attend(mixer, lengths, a.more)
    train(mixer, ("norm_weight", "norm_bias"), lengths)
    torch.cuda.synchronize()
    gdr.gdr_profile_enable(False)
    for name, (n, ms, _) in sorted(gdr.gdr_profile_report().items(), key=lambda kv: -kv[1][1]):
        print(f"  {name:14s} {n:5d} launches {1e3 * ms / n:9.2f} us each")
    return max(d, da), t


if __name__ == "__main__":
    main()
