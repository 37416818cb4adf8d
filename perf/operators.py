"""Measured cases of the block's RMS norm and gated feed-forward operators.

Two operators of the residual stream, each in its forms:

* the root-mean-square norm with the residual's addition: s = x + residual
  (stored in bf16), y = s / sqrt(mean(s^2) + eps) * gamma, y in bf16 ("rms")
  or in e4m3 with one scale a row ("rms_q8"), and its backward pass ("rms_bwd");
* the gated feed-forward block: y = residual + (act(x Wg^T + bg) * (x Wu^T +
  bu)) Wd^T + bd in bf16 ("gated"), with x, Wg and Wu in e4m3 with a scale a
  row ("gated_q8"), and its backward pass ("gated_bwd").

`own` false: the plain form, elementary torch operations in 32 bits.  `own`
true: the calls a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
DEV = "cuda"


def listed():
    return [
        # the next token of one sequence: latency of the norm between two sub-layers
        dict(name="rms_token", form="rms", rows=1, C=2048, residual=True),
        # Swin-T stage 1, a batch of 64 images of 56 x 56 tokens
        dict(name="rms_swin_t_s1", form="rms", rows=200704, C=96, residual=True),
        # a prompt one token short of 8 K, quantised for an 8-bit projection
        dict(name="rms_q8_prompt", form="rms_q8", rows=8191, C=4096, residual=True),
        # training on SwinV2-L's 4 x 384 x 384 tokens, the sum's own gradient added
        dict(name="rms_bwd_swinv2_l", form="rms_bwd", rows=589824, C=192, residual=True),
        # a ragged training batch at a width that is no power of two
        dict(name="rms_bwd_ragged", form="rms_bwd", rows=3001, C=2744, residual=False),
        # the next token of one sequence: the weights are read once for one row
        dict(name="gated_token", form="gated", rows=1, C=2048, F=5632, act="silu", bias=False, residual=True),
        # Swin-T stage 1: many tokens, small weights
        dict(name="gated_swin_t_s1", form="gated", rows=200704, C=96, F=256, act="gelu", bias=True, residual=True),
        # a long prompt through a wide layer: bound by the matrix products
        dict(name="gated_prompt", form="gated", rows=8192, C=2048, F=8192, act="silu", bias=False, residual=True),
        # the next tokens of 24 sequences, weights in 8 bits
        dict(name="gated_q8_batch", form="gated_q8", rows=24, C=4096, F=11264, act="silu", bias=False, residual=True),
        # a ragged prompt, widths that end inside a tile
        dict(name="gated_q8_ragged", form="gated_q8", rows=1537, C=1536, F=4104, act="silu", bias=True,
             residual=False),
        # training on Swin-B stage 3 (64 x 14 x 14 tokens), hidden width 8/3 C
        dict(name="gated_bwd_swin_b_s3", form="gated_bwd", rows=12544, C=512, F=1368, act="gelu", bias=True),
        # training on a packed batch of 4 K tokens
        dict(name="gated_bwd_prompt", form="gated_bwd", rows=4096, C=2048, F=5632, act="silu", bias=False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    form = rng.choice(["rms", "rms_q8", "rms_bwd", "gated", "gated_q8", "gated_bwd"])
    if form.startswith("rms"):
        C = 8 * int(_log(rng, 4, 1024))
        rows = int(_log(rng, 1, min(600000, 110e6 / C)))
        return dict(form=form, rows=rows, C=C, residual=rng.random() < 0.6)
    C = 16 * int(_log(rng, 4, 256)) + (8 if form != "gated_q8" and rng.random() < 0.5 else 0)
    F = min(16 * 1024, 8 * int(C * rng.uniform(1.0, 4.5) / 8))
    most = 825e9 / 6 if form != "gated_bwd" else 750e9 / 16
    rows = int(_log(rng, 1, min(200000, most / (C * F), 300e6 / F)))
    c = dict(form=form, rows=rows, C=C, F=F, act=rng.choice(["silu", "gelu"]), bias=rng.random() < 0.5)
    if form != "gated_bwd":
        c["residual"] = rng.random() < 0.6
    return c


def _quantise(w):
    """[n, k] fp32 -> e4m3 codes and the fp32 scale of each row."""
    s = w.abs().amax(1).clamp_min(1e-30) / E4M3_MAX
    return (w / s[:, None]).to(torch.float8_e4m3fn), s


class _Handle:
    """A library handle that is freed with the state that keeps it."""

    def __init__(self, case):
        from vision_transformer_shifted_gb300 import binding as sw
        if case["form"].startswith("rms"):
            self.h, self.free = sw.swin_block_rms_create(case["C"], EPS), sw.swin_block_rms_destroy
        else:
            act = sw.BLOCK_GATED_SILU if case["act"] == "silu" else sw.BLOCK_GATED_GELU
            self.h, self.free = sw.swin_block_gated_create(case["C"], case["F"], act), sw.swin_block_gated_destroy
        self.sw = sw

    def __del__(self):
        if getattr(self, "h", None) is not None:
            self.free(self.h)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)

    T, C, form = case["rows"], case["C"], case["form"]
    if form.startswith("rms"):
        d = dict(x=normal(T, C), gamma=(1 + 0.1 * torch.randn(C, generator=g, device=DEV)).to(bf))
        if T > 16:
            d["x"][-3:] = 0   # padding tokens behind the last sequence
        if form == "rms_bwd":
            d["dy"] = normal(T, C)
        d["residual"] = normal(T, C) if case["residual"] else None   # rms_bwd: the gradient that reaches the sum
        if case["residual"] and T > 16 and form != "rms_bwd":
            d["residual"][-3:] = 0
        return d
    F = case["F"]
    d = dict(x=normal(T, C), Wd=normal(C, F, std=F ** -0.5))
    for n in ("g", "u"):
        d["W" + n] = normal(F, C, std=C ** -0.5)
    for n, k in (("bg", F), ("bu", F), ("bd", C)):
        d[n] = normal(k, std=0.1) if case["bias"] else None
    if form == "gated_bwd":
        d["dy"] = normal(T, C)
        return d
    d["residual"] = normal(T, C) if case["residual"] else None
    if form == "gated_q8":
        d["x8"], d["sx"] = _quantise(d.pop("x").float())
        d["Wg8"], d["sg"] = _quantise(d.pop("Wg").float())
        d["Wu8"], d["su"] = _quantise(d.pop("Wu").float())
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    T, C, form, bf = case["rows"], case["C"], case["form"], torch.bfloat16
    new = lambda *s, t=bf: torch.empty(*s, device=DEV, dtype=t)  # noqa: E731
    out = {}
    if form in ("rms", "rms_q8"):
        out["sum"] = new(T, C) if case["residual"] else None
        if form == "rms":
            out["out"] = new(T, C)
        else:
            out["out8"], out["scales"] = new(T, C, t=torch.float8_e4m3fn), new(T, t=torch.float32)
    elif form == "rms_bwd":
        out["dx"], out["dgamma"] = new(T, C), new(C, t=torch.float32)
    elif form == "gated_bwd":
        out["dx"] = new(T, C)
        for n in ("Wg", "Wu", "Wd", "bg", "bu", "bd"):
            out["d" + n] = torch.empty_like(d[n]) if d[n] is not None else None
    else:
        out["out"] = new(T, C)
    return dict(case=case, d=d, out=out, handle=_Handle(case) if own else None)


def _run_own(case, d, o, handle):
    sw, h, form = handle.sw, handle.h, case["form"]
    if form == "rms":
        sw.swin_block_rms_forward(h, d["x"], d["gamma"], o["out"], residual=d["residual"], out_sum=o["sum"])
    elif form == "rms_q8":
        sw.swin_block_rms_forward_q8(h, d["x"], d["gamma"], o["out8"], o["scales"], residual=d["residual"],
                                     out_sum=o["sum"])
    elif form == "rms_bwd":
        sw.swin_block_rms_backward(h, d["x"], d["gamma"], d["dy"], o["dx"], o["dgamma"], dsum=d["residual"])
    elif form == "gated":
        sw.swin_block_gated_forward(h, d["x"], d, o["out"], residual=d["residual"])
    elif form == "gated_q8":
        sw.swin_block_gated_forward_q8(h, d["x8"], d["sx"], d, o["out"], residual=d["residual"])
    else:
        sw.swin_block_gated_backward(h, d["x"], d, d["dy"], o["dx"], o)
    return o


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    phi = 0.5 * (1 + torch.erf(g * 2 ** -0.5))
    return g * phi, phi + g * torch.exp(-0.5 * g * g) * (2 * math.pi) ** -0.5


def _linear(x, w, b):
    y = x @ w.t()
    return y if b is None else y + b.float()


def _rms_plain(case, d):
    s = d["x"]
    if case["residual"]:
        s = (s.float() + d["residual"].float()).to(torch.bfloat16)   # the stored sum is what is normalised
    sf = s.float()
    y = sf * torch.rsqrt((sf * sf).mean(1, keepdim=True) + EPS) * d["gamma"].float()
    o = dict(sum=s if case["residual"] else None)
    if case["form"] == "rms":
        o["out"] = y.to(torch.bfloat16)
    else:
        o["out8"], o["scales"] = _quantise(y)
    return o


def _rms_bwd_plain(d):
    s, dy, gamma = d["x"].float(), d["dy"].float(), d["gamma"].float()
    r = torch.rsqrt((s * s).mean(1, keepdim=True) + EPS)
    n = s * r
    a = dy * gamma
    dx = r * (a - n * (a * n).mean(1, keepdim=True))
    if d["residual"] is not None:
        dx = dx + d["residual"].float()
    return dict(dx=dx.to(torch.bfloat16), dgamma=(dy * n).sum(0))


def _gated_plain(case, d):
    if case["form"] == "gated":
        x, wg, wu = d["x"].float(), d["Wg"].float(), d["Wu"].float()
    else:
        x = d["x8"].float() * d["sx"][:, None]
        wg, wu = d["Wg8"].float() * d["sg"][:, None], d["Wu8"].float() * d["su"][:, None]
    h = _act(_linear(x, wg, d["bg"]), case["act"])[0] * _linear(x, wu, d["bu"])
    y = _linear(h, d["Wd"].float(), d["bd"])
    if case["residual"]:
        y = y + d["residual"].float()
    return dict(out=y.to(torch.bfloat16))


def _gated_bwd_plain(case, d):
    bf = torch.bfloat16
    x, dy, wg, wu, wd = (d[n].float() for n in ("x", "dy", "Wg", "Wu", "Wd"))
    g, u = _linear(x, wg, d["bg"]), _linear(x, wu, d["bu"])
    a, da = _act(g, case["act"])
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    o = dict(dx=(dg @ wg + du @ wu).to(bf), dWg=(dg.t() @ x).to(bf), dWu=(du.t() @ x).to(bf),
             dWd=(dy.t() @ (a * u)).to(bf), dbg=None, dbu=None, dbd=None)
    if case["bias"]:
        o["dbg"], o["dbu"], o["dbd"] = dg.sum(0).to(bf), du.sum(0).to(bf), dy.sum(0).to(bf)
    return o


def run(state):
    case, d = state["case"], state["d"]
    if own:
        return _run_own(case, d, state["out"], state["handle"])
    if case["form"] in ("rms", "rms_q8"):
        return _rms_plain(case, d)
    if case["form"] == "rms_bwd":
        return _rms_bwd_plain(d)
    if case["form"] == "gated_bwd":
        return _gated_bwd_plain(case, d)
    return _gated_plain(case, d)


def work(case):
    T, C, form = case["rows"], case["C"], case["form"]
    if form in ("rms", "rms_q8"):
        rows = 2 * T * C * (3 if case["residual"] else 1) + 2 * C   # x, residual and sum
        return dict(bytes=rows + (2 * T * C if form == "rms" else T * C + 4 * T), flops=5 * T * C)
    if form == "rms_bwd":
        return dict(bytes=2 * T * C * (4 if case["residual"] else 3) + 6 * C, flops=10 * T * C)
    F = case["F"]
    if form == "gated_bwd":
        return dict(bytes=6 * T * C + 12 * C * F + (4 * (2 * F + C) if case["bias"] else 0), flops=16 * T * C * F)
    wide = 1 if form == "gated_q8" else 2
    by = T * C * (wide + 2 + (2 if case["residual"] else 0)) + 2 * C * F * wide + 2 * C * F
    if form == "gated_q8":
        by += 4 * T + 8 * F
    return dict(bytes=by + (2 * (2 * F + C) if case["bias"] else 0), flops=6 * T * C * F)


def exact(case, seed):
    d, form = _inputs(case, seed), case["form"]
    D = lambda n: d[n].double()  # noqa: E731
    if form == "rms_bwd":
        ms = D("x").pow(2).mean(-1) + EPS
        w = torch.einsum("tc,c,tc->t", D("dy"), D("gamma"), D("x")) / case["C"]
        dx = D("dy") * D("gamma") / ms.sqrt()[:, None] - D("x") * (w / ms ** 1.5)[:, None]
        if case["residual"]:
            dx += D("residual")
        return dict(dx=dx, dgamma=torch.einsum("tc,tc,t->c", D("dy"), D("x"), ms ** -0.5))
    if form.startswith("rms"):
        s = total = D("x")
        if case["residual"]:
            total = s + D("residual")
            s = total.to(torch.bfloat16).double()
        y = s / (s.pow(2).mean(-1) + EPS).sqrt()[:, None] * D("gamma")
        o = dict(sum=total if case["residual"] else None)
        if form == "rms":
            o["out"] = y
        else:
            o["scales"] = y.abs().amax(-1).clamp_min(1e-30) / E4M3_MAX
            o["out8"] = y / o["scales"][:, None]
        return o
    if form == "gated_q8":
        x, wg, wu = (D(w) * D(s)[:, None] for w, s in (("x8", "sx"), ("Wg8", "sg"), ("Wu8", "su")))
    else:
        x, wg, wu = D("x"), D("Wg"), D("Wu")
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    b = {n: D(n) if d[n] is not None else zero for n in ("bg", "bu", "bd")}
    g = torch.einsum("tc,fc->tf", x, wg) + b["bg"]
    u = torch.einsum("tc,fc->tf", x, wu) + b["bu"]
    gate = torch.sigmoid(g) if case["act"] == "silu" else torch.special.ndtr(g)   # act(g) = g gate(g)
    if form != "gated_bwd":
        y = torch.einsum("tf,cf->tc", g * gate * u, D("Wd")) + b["bd"]
        return dict(out=y + D("residual") if case["residual"] else y)
    slope = gate * (1 - gate) if case["act"] == "silu" else (-g * g / 2).exp() / (2 * math.pi) ** 0.5
    dh = torch.einsum("tc,cf->tf", D("dy"), D("Wd"))
    du = dh * g * gate
    dg = dh * u * (gate + g * slope)
    bias = case["bias"]
    return dict(dx=torch.einsum("tf,fc->tc", dg, wg) + torch.einsum("tf,fc->tc", du, wu),
                dWg=torch.einsum("tf,tc->fc", dg, x), dWu=torch.einsum("tf,tc->fc", du, x),
                dWd=torch.einsum("tc,tf->cf", D("dy"), g * gate * u), dbg=dg.sum(0) if bias else None,
                dbu=du.sum(0) if bias else None, dbd=D("dy").sum(0) if bias else None)
