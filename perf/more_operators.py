"""Measured cases of the block's layer norm and linear operators.

Two operators that training and serving a block need beside its attention, each
in its forms:

* the layer norm of the residual stream: s = x + residual (stored in bf16),
  y = (s - mean) / sqrt(var + eps) * gamma + beta, y in bf16 ("ln") or in e4m3
  with one scale a row ("ln_q8"); the residual post-norm y = residual +
  LN(x) ("ln_post"); the backward pass of them all ("ln_bwd");
* the matrix product with its epilogue: z = x W^T + b, y = residual + act(z) in
  bf16 ("linear"; z kept for training), with x and W in e4m3, a scale a row
  ("linear_q8"), and its backward pass ("linear_bwd").

`own` false: the plain form, elementary torch operations in 32 bits.  `own`
true: the calls a user makes of the library.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3_MAX = 448.0
DEV = "cuda"


def listed():
    return [
        # the next token of one sequence: latency of the norm between two sub-layers
        dict(name="ln_token", form="ln", rows=1, C=2048, residual=True),
        # Swin-T stage 1 (64 images of 56 x 56 tokens), between attention and MLP
        dict(name="ln_swin_t_s1", form="ln", rows=200704, C=96, residual=True),
        # SwinV2-L's 4 x 384 x 384 tokens: each branch is normalised before it is added
        dict(name="ln_post_swinv2_l", form="ln_post", rows=589824, C=192, residual=True),
        # a prompt one token short of 8 K, quantised for an 8-bit projection
        dict(name="ln_q8_prompt", form="ln_q8", rows=8191, C=4096, residual=True),
        # training on SwinV2-L's tokens, the sum's own gradient added
        dict(name="ln_bwd_swinv2_l", form="ln_bwd", rows=589824, C=192, residual=True),
        # a ragged training batch at a width that is no power of two
        dict(name="ln_bwd_ragged", form="ln_bwd", rows=3001, C=2744, residual=False),
        # the next token of one sequence: the weights are read once for one row
        dict(name="linear_token", form="linear", rows=1, C=2048, N=8192, act="gelu", bias=True, residual=False,
             keep=False),
        # the next tokens of 24 sequences, weights in 8 bits
        dict(name="linear_q8_batch", form="linear_q8", rows=24, C=4096, N=11264, act="silu", bias=True,
             residual=False),
        # training, Swin-T stage 1: the MLP's first layer, its pre-activation kept
        dict(name="linear_swin_t_s1", form="linear", rows=200704, C=96, N=384, act="gelu", bias=True, residual=False,
             keep=True),
        # a long prompt through a wide layer's second product: bound by the matrix products
        dict(name="linear_prompt", form="linear", rows=8192, C=8192, N=2048, act="none", bias=True, residual=True,
             keep=False),
        # training, Swin-B stage 3 (64 x 14 x 14 tokens): the MLP's first layer
        dict(name="linear_bwd_swin_b_s3", form="linear_bwd", rows=12544, C=512, N=2048, act="gelu", bias=True),
        # training on a packed batch that ends one token past 4 K: a projection without activation
        dict(name="linear_bwd_prompt", form="linear_bwd", rows=4097, C=2048, N=5632, act="none", bias=False),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    form = rng.choice(["ln", "ln_post", "ln_q8", "ln_bwd", "linear", "linear", "linear_q8", "linear_bwd"])
    if form.startswith("ln"):
        C = 8 * int(_log(rng, 4, 1024))
        rows = int(_log(rng, 1, min(600000, 110e6 / C)))
        return dict(form=form, rows=rows, C=C, residual=form == "ln_post" or rng.random() < 0.6)
    eighths = 0 if form == "linear_q8" else 8 * int(rng.random() < 0.5)
    C = 16 * int(_log(rng, 4, 500)) + eighths
    N = 8 * int(_log(rng, 8, 1400))
    most = 270e9 / 2 if form != "linear_bwd" else 185e9 / 4
    rows = int(_log(rng, 1, min(200000, most / (C * N), 75e6 / max(C, N))))
    c = dict(form=form, rows=rows, C=C, N=N, act=rng.choice(["none", "silu", "gelu"]), bias=rng.random() < 0.6)
    if form != "linear_bwd":
        c["residual"] = rng.random() < 0.5
    if form == "linear":
        c["keep"] = c["act"] != "none" and rng.random() < 0.5
    return c


def _quantise(w):
    """[n, k] fp32 -> e4m3 codes and the fp32 scale of each row."""
    s = w.abs().amax(1).clamp_min(1e-30) / E4M3_MAX
    return (w / s[:, None]).to(torch.float8_e4m3fn), s


class _Handle:
    """A library handle that is freed with the state that keeps it."""

    def __init__(self, case):
        from vision_transformer_shifted_gb300 import binding as sw
        if case["form"].startswith("ln"):
            self.h, self.free = sw.swin_block_layernorm_create(case["C"], EPS), sw.swin_block_layernorm_destroy
        else:
            act = dict(none=sw.BLOCK_LINEAR_NONE, silu=sw.BLOCK_LINEAR_SILU, gelu=sw.BLOCK_LINEAR_GELU)[case["act"]]
            self.h, self.free = sw.swin_block_linear_create(case["C"], case["N"], act), sw.swin_block_linear_destroy
        self.sw = sw

    def __del__(self):
        if getattr(self, "h", None) is not None:
            self.free(self.h)


def _inputs(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, mean=0.0, dtype=bf):
        return (torch.randn(*shape, generator=g, device=DEV) * std + mean).to(dtype)

    T, C, form = case["rows"], case["C"], case["form"]
    if form.startswith("ln"):
        # a residual stream: every channel has a mean of its own, a few are large
        centre = torch.randn(C, generator=g, device=DEV) * 0.5
        centre[::64] *= 16
        d = dict(x=(torch.randn(T, C, generator=g, device=DEV) + centre).to(bf), gamma=normal(C, std=0.1, mean=1.0),
                 beta=normal(C, std=0.1))
        d["residual"] = normal(T, C) if case["residual"] else None   # ln_bwd: the gradient that reaches the sum
        if form == "ln_bwd":
            d["dy"] = normal(T, C)
        if T > 16:
            for n in ("x", "residual", "dy"):
                if d.get(n) is not None:
                    d[n][-3:] = 0   # padding tokens behind the last sequence
        return d
    N = case["N"]
    d = dict(x=normal(T, C), W=normal(N, C, std=C ** -0.5), b=normal(N, std=0.1) if case["bias"] else None)
    if form == "linear_bwd":
        d["dy"], d["z"] = normal(T, N), None
        if case["act"] != "none":
            z = d["x"] @ d["W"].t()
            d["z"] = z if d["b"] is None else z + d["b"]
        return d
    d["residual"] = normal(T, N) if case["residual"] else None
    if form == "linear_q8":
        d["x8"], d["sx"] = _quantise(d.pop("x").float())
        d["W8"], d["sw"] = _quantise(d.pop("W").float())
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    T, C, form, bf = case["rows"], case["C"], case["form"], torch.bfloat16
    new = lambda *s, t=bf: torch.empty(*s, device=DEV, dtype=t)  # noqa: E731
    out = {}
    if form in ("ln", "ln_q8"):
        out["sum"] = new(T, C) if case["residual"] else None
    if form in ("ln", "ln_post"):
        out["out"] = new(T, C)
    elif form == "ln_q8":
        out["out8"], out["scales"] = new(T, C, t=torch.float8_e4m3fn), new(T, t=torch.float32)
    elif form == "ln_bwd":
        out["dx"], out["dgamma"], out["dbeta"] = new(T, C), new(C, t=torch.float32), new(C, t=torch.float32)
    elif form == "linear_bwd":
        out["dx"], out["dW"] = new(T, C), new(case["N"], C)
        out["db"] = new(case["N"]) if case["bias"] else None
    else:
        out["out"] = new(T, case["N"])
        if form == "linear":
            out["z"] = new(T, case["N"]) if case["keep"] else None
    return dict(case=case, d=d, out=out, handle=_Handle(case) if own else None)


def _run_own(case, d, o, handle):
    sw, h, form = handle.sw, handle.h, case["form"]
    if form == "ln":
        sw.swin_block_layernorm_forward(h, d["x"], d["gamma"], d["beta"], o["out"], residual=d["residual"],
                                        out_sum=o["sum"])
    elif form == "ln_post":
        sw.swin_block_layernorm_forward_post(h, d["x"], d["gamma"], d["beta"], d["residual"], o["out"])
    elif form == "ln_q8":
        sw.swin_block_layernorm_forward_q8(h, d["x"], d["gamma"], d["beta"], o["out8"], o["scales"],
                                           residual=d["residual"], out_sum=o["sum"])
    elif form == "ln_bwd":
        sw.swin_block_layernorm_backward(h, d["x"], d["gamma"], d["dy"], o["dx"], o["dgamma"], o["dbeta"],
                                         dsum=d["residual"])
    elif form == "linear":
        sw.swin_block_linear_forward(h, d["x"], d["W"], d["b"], o["out"], residual=d["residual"], z=o["z"])
    elif form == "linear_q8":
        sw.swin_block_linear_forward_q8(h, d["x8"], d["sx"], d["W8"], d["sw"], d["b"], o["out"],
                                        residual=d["residual"])
    else:
        sw.swin_block_linear_backward(h, d["x"], d["W"], d["dy"], o["dx"], o["dW"], o["db"], z=d["z"])
    return o


def _normalised(s):
    """The normalised rows and 1 / sqrt(var + eps), 32 bits."""
    c = s - s.mean(1, keepdim=True)
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    return c * r, r


def _ln_plain(case, d):
    s, form = d["x"], case["form"]
    if case["residual"] and form != "ln_post":
        s = (s.float() + d["residual"].float()).to(torch.bfloat16)   # the stored sum is what is normalised
    y = _normalised(s.float())[0] * d["gamma"].float() + d["beta"].float()
    if form == "ln_post":
        return dict(out=(d["residual"].float() + y).to(torch.bfloat16))
    o = dict(sum=s if case["residual"] else None)
    if form == "ln":
        o["out"] = y.to(torch.bfloat16)
    else:
        o["out8"], o["scales"] = _quantise(y)
    return o


def _ln_bwd_plain(d):
    dy = d["dy"].float()
    n, r = _normalised(d["x"].float())
    a = dy * d["gamma"].float()
    dx = r * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
    if d["residual"] is not None:
        dx = dx + d["residual"].float()
    return dict(dx=dx.to(torch.bfloat16), dgamma=(dy * n).sum(0), dbeta=dy.sum(0))


def _act(z, act):
    """The activation and its derivative."""
    if act == "none":
        return z, 1.0
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    phi = 0.5 * (1 + torch.erf(z * 2 ** -0.5))
    return z * phi, phi + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5


def _linear_plain(case, d):
    if case["form"] == "linear":
        x, w = d["x"].float(), d["W"].float()
    else:
        x, w = d["x8"].float() * d["sx"][:, None], d["W8"].float() * d["sw"][:, None]
    z = x @ w.t()
    if d["b"] is not None:
        z = z + d["b"].float()
    y = _act(z, case["act"])[0]
    if case["residual"]:
        y = y + d["residual"].float()
    o = dict(out=y.to(torch.bfloat16))
    if case["form"] == "linear":
        o["z"] = z.to(torch.bfloat16) if case["keep"] else None
    return o


def _linear_bwd_plain(case, d):
    bf = torch.bfloat16
    dz = d["dy"].float()
    if case["act"] != "none":
        dz = dz * _act(d["z"].float(), case["act"])[1]
    return dict(dx=(dz @ d["W"].float()).to(bf), dW=(dz.t() @ d["x"].float()).to(bf),
                db=dz.sum(0).to(bf) if case["bias"] else None)


def run(state):
    case, d = state["case"], state["d"]
    if own:
        return _run_own(case, d, state["out"], state["handle"])
    if case["form"] == "ln_bwd":
        return _ln_bwd_plain(d)
    if case["form"] == "linear_bwd":
        return _linear_bwd_plain(case, d)
    return (_ln_plain if case["form"].startswith("ln") else _linear_plain)(case, d)


def work(case):
    T, C, form = case["rows"], case["C"], case["form"]
    if form == "ln_bwd":
        return dict(bytes=2 * T * C * (4 if case["residual"] else 3) + 10 * C, flops=14 * T * C)
    if form == "ln_post":
        return dict(bytes=6 * T * C + 4 * C, flops=8 * T * C)
    if form in ("ln", "ln_q8"):
        rows = 2 * T * C * (3 if case["residual"] else 1) + 4 * C   # x, residual and sum
        return dict(bytes=rows + (2 * T * C if form == "ln" else T * C + 4 * T), flops=8 * T * C)
    N = case["N"]
    if form == "linear_bwd":
        by = 4 * T * C + 4 * C * N + 2 * T * N * (1 if case["act"] == "none" else 2)
        return dict(bytes=by + (2 * N if case["bias"] else 0), flops=4 * T * C * N)
    wide = 1 if form == "linear_q8" else 2
    by = wide * (T * C + C * N) + 2 * T * N * (1 + bool(case["residual"]) + bool(case.get("keep")))
    if form == "linear_q8":
        by += 4 * T + 4 * N
    return dict(bytes=by + (2 * N if case["bias"] else 0), flops=2 * T * C * N)


def exact(case, seed):
    d, form = _inputs(case, seed), case["form"]
    D = lambda n: d[n].double()  # noqa: E731
    if form.startswith("ln"):
        s = total = D("x")
        if case["residual"] and form in ("ln", "ln_q8"):
            total = s + D("residual")
            s = total.to(torch.bfloat16).double()
        var, mean = torch.var_mean(s, 1, correction=0, keepdim=True)
        sd = (var + EPS).sqrt()
        if form == "ln_bwd":
            n = (s - mean) / sd
            a = torch.einsum("tc,c->tc", D("dy"), D("gamma"))
            dx = (a - (a.sum(1, keepdim=True) + n * torch.einsum("tc,tc->t", a, n)[:, None]) / case["C"]) / sd
            if case["residual"]:
                dx += D("residual")
            return dict(dx=dx, dgamma=torch.einsum("tc,tc->c", D("dy"), n), dbeta=D("dy").sum(0))
        y = torch.addcmul(D("beta"), (s - mean) / sd, D("gamma"))
        if form == "ln_post":
            return dict(out=D("residual") + y)
        o = dict(sum=total if case["residual"] else None)
        if form == "ln":
            o["out"] = y
        else:
            o["scales"] = y.abs().amax(-1).clamp_min(1e-30) / E4M3_MAX
            o["out8"] = y / o["scales"][:, None]
        return o
    if form == "linear_bwd":
        dz = D("dy")
        if case["act"] != "none":
            z = D("z")
            gate = torch.sigmoid(z) if case["act"] == "silu" else torch.special.ndtr(z)   # act(z) = z gate(z)
            slope = gate * (1 - gate) if case["act"] == "silu" else (-z * z / 2).exp() / (2 * math.pi) ** 0.5
            dz = dz * (gate + z * slope)
        return dict(dx=torch.einsum("tn,nc->tc", dz, D("W")), dW=torch.einsum("tn,tc->nc", dz, D("x")),
                    db=dz.sum(0) if case["bias"] else None)
    if form == "linear_q8":
        x, w = D("x8") * D("sx")[:, None], D("W8") * D("sw")[:, None]
    else:
        x, w = D("x"), D("W")
    z = torch.einsum("tc,nc->tn", x, w)
    if d["b"] is not None:
        z += D("b")
    y = dict(none=lambda: z, silu=lambda: z * torch.sigmoid(z), gelu=lambda: z * torch.special.ndtr(z))[case["act"]]()
    o = dict(out=y + D("residual") if case["residual"] else y)
    if form == "linear":
        o["z"] = z if case["keep"] else None
    return o
