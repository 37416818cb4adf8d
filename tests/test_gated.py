"""Gated feed-forward block (include/swin_gated.h).

CPU (not gpu): refusals, and the gradient formulas against autograd in
float64 and against differences.  GPU: forward (bf16, 8-bit) and backward
against the formulas in float64, at sizes on each side of the kernels' tiles
and plans (one row, tiles that end inside, K slices, several products in one
launch), biases and residuals present or not, in place, on two streams,
captured and replayed, and the run norm -> gated block -> norm with its
backward.

Tolerances: every stored bf16 value is off by at most 2^-8 of itself.  out =
h Wd^T with h stored in bf16: |error| <= 2^-8 |out| + sum_f (2^-8 |h| + 2^-17
|u| (1 + |g|)) |Wd| (the last term: the activation in fp32, an erf good to
5.5e-7, and the fp32 sums g and u); the same for the products that read dg
and du.  Those are worst cases, so the relative error in the 2-norm is held
too: two roundings of at most 2^-8 each, the inner one averaged over a sum.
"""
import ctypes
import os

import pytest
import torch

from vision_transformer_shifted_gb300 import binding as sw

DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = 2.0 ** -8
ACTS = {"silu": sw.BLOCK_GATED_SILU, "gelu": sw.BLOCK_GATED_GELU}


def act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    phi = torch.special.ndtr(g)
    return g * phi, phi + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5


def lin(x, w, b):
    y = x @ w.t()
    return y if b is None else y + b


def forward_ref(x, p, residual, kind):
    """out and the bound on its error (float64)."""
    d = {k: None if v is None else v.double() for k, v in p.items()}
    x = x.double()
    g, u = lin(x, d["Wg"], d["bg"]), lin(x, d["Wu"], d["bu"])
    h = act(g, kind)[0] * u
    out = lin(h, d["Wd"], d["bd"])
    if residual is not None:
        out = out + residual.double()
    inner = HALF * h.abs() + 2.0 ** -17 * u.abs() * (1 + g.abs())
    return out, HALF * 1.01 * out.abs() + inner @ d["Wd"].abs().t()


def backward_ref(x, p, dy, kind):
    """Gradients and the bounds on their errors (float64)."""
    d = {k: None if v is None else v.double() for k, v in p.items()}
    x, dy = x.double(), dy.double()
    g, u = lin(x, d["Wg"], d["bg"]), lin(x, d["Wu"], d["bu"])
    a, da = act(g, kind)
    dh = dy @ d["Wd"]
    dg, du, h = dh * u * da, dh * a, a * u
    small = 2.0 ** -17 * (1 + g.abs())
    eg = HALF * dg.abs() + small * (dh * u).abs()
    eu = HALF * du.abs() + small * dh.abs()
    eh = HALF * h.abs() + small * u.abs()
    ref = dict(dx=dg @ d["Wg"] + du @ d["Wu"], dWg=dg.t() @ x, dWu=du.t() @ x, dWd=dy.t() @ h, dbg=dg.sum(0),
               dbu=du.sum(0), dbd=dy.sum(0))
    err = dict(dx=eg @ d["Wg"].abs() + eu @ d["Wu"].abs(), dWg=eg.t() @ x.abs(), dWu=eu.t() @ x.abs(),
               dWd=dy.abs().t() @ eh, dbg=eg.sum(0), dbu=eu.sum(0), dbd=2.0 ** -17 * dy.abs().sum(0))
    return ref, {k: HALF * 1.01 * ref[k].abs() + err[k] for k in ref}


def close(got, ref, tol, rel=2 * HALF):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= tol + 1e-30).all(), float((err - tol).max())
    if ref.numel() >= 64:   # (a norm of many roundings)
        assert float(err.norm() / ref.norm()) <= rel


def make(rows, C, F, bias=True, residual=True, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + C * 17 + F)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    p = dict(Wg=n(F, C, std=C ** -0.5), Wu=n(F, C, std=C ** -0.5), Wd=n(C, F, std=F ** -0.5))
    for k, m in (("bg", F), ("bu", F), ("bd", C)):
        p[k] = n(m, std=0.3) if bias else None
    return n(rows, C), p, n(rows, C) if residual else None, n(rows, C)


def dev(p):
    if isinstance(p, dict):
        return {k: dev(v) for k, v in p.items()}
    return None if p is None else p.to(DEV)


def quantise(w):
    s = w.float().abs().amax(-1).clamp_min(1e-30) / 448
    return (w.float() / s[:, None]).to(E4M3), s


class gated:
    def __init__(self, C, F, kind="silu"):
        self.args = C, F, ACTS[kind]

    def __enter__(self):
        self.h = sw.swin_block_gated_create(*self.args)
        return self.h

    def __exit__(self, *exc):
        sw.swin_block_gated_destroy(self.h)


def new_grads(p, dev=DEV):
    return {"d" + k: None if v is None else torch.full(v.shape, float("nan"), dtype=BF, device=dev)
            for k, v in p.items()}


# ---- CPU ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_formulas(kind):
    g = torch.Generator().manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    T, C, F = 5, 8, 16
    x, dy = n(T, C), n(T, C)
    p = dict(Wg=n(F, C) * 0.4, bg=n(F), Wu=n(F, C) * 0.4, bu=n(F), Wd=n(C, F) * 0.3, bd=n(C))

    def loss(x, p):
        a = lin(x, p["Wg"], p["bg"])
        a = torch.nn.functional.silu(a) if kind == "silu" else torch.nn.functional.gelu(a)
        return (lin(a * lin(x, p["Wu"], p["bu"]), p["Wd"], p["bd"]) * dy).sum()

    ref, _ = backward_ref(x, p, dy, kind)
    leaves = {k: v.clone().requires_grad_() for k, v in dict(p, x=x).items()}
    loss(leaves["x"], leaves).backward()
    for k, t in leaves.items():
        assert torch.allclose(ref["d" + k], t.grad, rtol=1e-12, atol=1e-12), k
        i = 3 % t.numel()   # and one entry each against a central difference
        e = torch.zeros(t.numel(), dtype=torch.float64)
        e[i] = 1e-5
        e = e.view(t.shape)
        args = dict(p, x=x)
        up, down = dict(args, **{k: args[k] + e}), dict(args, **{k: args[k] - e})
        diff = float(loss(up["x"], up) - loss(down["x"], down)) / 2e-5
        assert abs(diff - float(ref["d" + k].reshape(-1)[i])) < 1e-6 * (1 + abs(diff)), k


@pytest.mark.parametrize("C,F,kind", [(0, 64, 0), (12, 64, 0), (64, 0, 0), (64, 12, 0), (-8, 64, 0), (65544, 64, 0),
                                      (64, 65544, 0), (64, 64, 2), (64, 64, -1)])
def test_create_refuses(C, F, kind):
    h = ctypes.c_void_p(1)
    assert sw.load().swin_block_gated_create(ctypes.byref(h), C, F, kind) == sw.EINVAL
    assert h.value is None
    assert sw.load().swin_block_gated_create(None, 64, 64, 0) == sw.EINVAL


P = 1 << 24   # addresses that no refused call reads
STEP = 1 << 16


def _addresses(names):
    return {n: P + i * STEP for i, n in enumerate(names)}


def test_forward_refuses():
    lib = sw.load()
    ok = _addresses(["Wg", "bg", "Wu", "bu", "Wd", "bd", "x", "residual", "out", "sx", "sg", "su"])

    def call(q8, rows=4, C=64, params=True, **kw):
        a = {**ok, **kw}
        with gated(C, 64) as h:
            h = a.get("h", h)
            if q8:
                s = sw.GatedParamsQ8(a["Wg"], a["sg"], a["bg"], a["Wu"], a["su"], a["bu"], a["Wd"], a["bd"])
                return lib.swin_block_gated_forward_q8(h, a["x"], a["sx"], rows,
                                                       ctypes.addressof(s) if params else None, a["residual"],
                                                       a["out"], None)
            s = sw.GatedParams(*(a[n] for n in ("Wg", "bg", "Wu", "bu", "Wd", "bd")))
            return lib.swin_block_gated_forward(h, a["x"], rows, ctypes.addressof(s) if params else None,
                                                a["residual"], a["out"], None)

    both = [dict(h=None), dict(params=False), dict(rows=-1)]
    both += [{n: None} for n in ("Wg", "Wu", "Wd", "x", "out")]
    both += [{n: ok[n] + 8} for n in ("Wg", "bg", "Wu", "bu", "Wd", "bd", "x", "residual", "out")]
    both += [dict(out=ok[n]) for n in ("Wg", "bg", "Wu", "bu", "Wd", "bd", "x")]
    both += [dict(out=ok["residual"] + 16), dict(rows=(1 << 31) - 1)]
    for bad in both:
        assert call(False, **bad) == sw.EINVAL, bad
        assert call(True, **bad) == sw.EINVAL, bad
    for bad in [{n: None} for n in ("sx", "sg", "su")] + [{n: ok[n] + 4} for n in ("sx", "sg", "su")] + [
            dict(out=ok[n]) for n in ("sx", "sg", "su")]:
        assert call(True, **bad) == sw.EINVAL, bad
    assert call(False, rows=0) == sw.OK and call(True, rows=0) == sw.OK
    assert call(True, C=72) == sw.EUNSUPPORTED
    assert lib.swin_block_gated_destroy(None) == sw.OK
    assert lib.swin_block_gated_last_launches(None) == 0
    assert lib.swin_block_gated_sync_status(None, None) == sw.EINVAL


def test_backward_refuses():
    lib = sw.load()
    ps, gs = ["Wg", "bg", "Wu", "bu", "Wd", "bd"], ["dWg", "dbg", "dWu", "dbu", "dWd", "dbd"]
    ok = _addresses(ps + gs + ["x", "dy", "dx"])

    def call(rows=4, params=True, grads=True, **kw):
        a = {**ok, **kw}
        s, g = sw.GatedParams(*(a[n] for n in ps)), sw.GatedParams(*(a[n] for n in gs))
        with gated(64, 64) as h:
            return lib.swin_block_gated_backward(a.get("h", h), a["x"], rows, ctypes.addressof(s) if params else None,
                                                 a["dy"], a["dx"], ctypes.addressof(g) if grads else None, None)

    bad = [dict(h=None), dict(params=False), dict(grads=False), dict(rows=-1), dict(rows=(1 << 31) - 1)]
    bad += [{n: None} for n in ("Wg", "Wu", "Wd", "x", "dy", "dx", "dWg", "dWu", "dWd")]
    bad += [{n: ok[n] + 2} for n in ok]
    bad += [{o: ok[i]} for o in gs + ["dx"] for i in ps + ["x", "dy"]]
    bad += [dict(dWg=ok["dWu"]), dict(dWd=ok["dx"]), dict(dbg=ok["dbu"]), dict(dbd=ok["dWd"])]
    for b in bad:
        assert call(**b) == sw.EINVAL, b


def test_binding_refuses_other_types_shapes_and_devices():
    x, p, r, _ = make(4, 64, 128)
    with gated(64, 128) as h:
        out = torch.empty_like(x)
        for kw in (dict(Wg=p["Wg"].float()), dict(Wd=p["Wd"].t().contiguous()), dict(bu=p["bu"][:64]), {}):
            with pytest.raises(ValueError):
                sw.swin_block_gated_forward(h, x, dict(p, **kw), out)
    x, p, r, _ = make(4, 64, 64)
    with gated(64, 128) as h, pytest.raises(ValueError):
        sw.swin_block_gated_forward(h, x, p, out)


# ---- GPU ---------------------------------------------------------------------------

SHAPES = [   # rows, C, F
    (1, 8, 8), (1, 96, 256), (1, 512, 1368), (2, 64, 64), (5, 136, 120), (17, 128, 264), (24, 1024, 2048),
    (64, 256, 640), (127, 192, 512), (128, 96, 128), (129, 328, 136), (256, 512, 512), (300, 1032, 2056),
    (515, 128, 384), (1000, 64, 1024), (3001, 96, 256), (2048, 768, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward(rows, C, F, kind):
    extra = kind == "silu"
    x, p, r, _ = make(rows, C, F, bias=extra, residual=extra)
    ref, tol = forward_ref(x, p, r, kind)
    out = torch.full((rows, C), float("nan"), dtype=BF, device=DEV)
    with gated(C, F, kind) as h:
        sw.swin_block_gated_forward(h, dev(x), dev(p), out, residual=dev(r))
        sw.swin_block_gated_sync_status(h)
    close(out, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [(129, 8, 8), (257, 120, 64), (300, 64, 72), (1000, 128, 576), (20000, 8, 136),
                                      (45001, 96, 256), (40000, 128, 200), (60001, 64, 64), (59000, 40, 328)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_narrow(rows, C, F, kind):
    """The one-kernel form: one chunk of hidden units, odd and even counts of
    them, weights that stay and weights that stream, several tiles a pair."""
    extra = (rows % 2 == 1) == (kind == "silu")
    x, p, r, _ = make(rows, C, F, bias=extra, residual=not extra, seed=9)
    ref, tol = forward_ref(x, p, r, kind)
    out = torch.full((rows, C), float("nan"), dtype=BF, device=DEV)
    with gated(C, F, kind) as h:
        sw.swin_block_gated_forward(h, dev(x), dev(p), out, residual=dev(r))
        sw.swin_block_gated_sync_status(h)
        assert sw.swin_block_gated_last_launches(h) == 1
    close(out, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [s for s in SHAPES if s[1] % 16 == 0])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_forward_q8(rows, C, F, kind):
    extra = kind == "gelu"
    x, p, r, _ = make(rows, C, F, bias=extra, residual=extra, seed=1)
    x8, sx = quantise(x)
    q = dict(bg=p["bg"], bu=p["bu"], Wd=p["Wd"], bd=p["bd"])
    (q["Wg8"], q["sg"]), (q["Wu8"], q["su"]) = quantise(p["Wg"]), quantise(p["Wu"])
    exact = dict(p, Wg=q["Wg8"].double() * q["sg"].double()[:, None], Wu=q["Wu8"].double() * q["su"].double()[:, None])
    ref, tol = forward_ref(x8.double() * sx.double()[:, None], exact, r, kind)
    out = torch.full((rows, C), float("nan"), dtype=BF, device=DEV)
    with gated(C, F, kind) as h:
        sw.swin_block_gated_forward_q8(h, dev(x8), dev(sx), dev(q), out, residual=dev(r))
        sw.swin_block_gated_sync_status(h)
    close(out, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", SHAPES)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_backward(rows, C, F, kind):
    x, p, _, dy = make(rows, C, F, bias=kind == "silu", seed=2)
    ref, tol = backward_ref(x, p, dy, kind)
    dx, grads = torch.full((rows, C), float("nan"), dtype=BF, device=DEV), new_grads(p)
    xd, pd, yd = dev(x), dev(p), dev(dy)
    with gated(C, F, kind) as h:
        sw.swin_block_gated_backward(h, xd, pd, yd, dx, grads)
        sw.swin_block_gated_sync_status(h)
        again, gagain = torch.empty_like(dx), new_grads(p)
        sw.swin_block_gated_backward(h, xd, pd, yd, again, gagain)
        sw.swin_block_gated_sync_status(h)
    for k, v in dict(grads, dx=dx).items():
        if v is not None:
            close(v, ref[k], tol[k])
            assert torch.equal(v, dict(gagain, dx=again)[k]), k   # sums in a fixed order


@pytest.mark.gpu
def test_large_values_and_nan_rows_stay_in_their_rows():
    """Gates far out on both sides of zero, and a row of NaN and one of
    infinities: only those rows are not finite."""
    rows, C, F = 140, 128, 256
    x, p, r, _ = make(rows, C, F, seed=3)
    x = (x.float() * 40).to(BF)
    x[7], x[130, 3] = float("nan"), float("inf")
    good = [i for i in range(rows) if i not in (7, 130)]
    for kind in ACTS:
        ref, tol = forward_ref(x[good], p, r[good], kind)
        out = torch.zeros(rows, C, dtype=BF, device=DEV)
        with gated(C, F, kind) as h:
            sw.swin_block_gated_forward(h, dev(x), dev(p), out, residual=dev(r))
            sw.swin_block_gated_sync_status(h)
        close(out[good], ref, tol)
        assert out[7].isnan().all() and not out[130].isfinite().any()


@pytest.mark.gpu
def test_in_place_and_rows_behind_the_batch():
    rows, C, F = 77, 192, 512
    x, p, r, dy = make(128, C, F, seed=4)
    xd, pd, rd, yd = dev(x), dev(p), dev(r), dev(dy)
    ref, tol = forward_ref(x[:rows], p, r[:rows], "silu")
    dx, grads = torch.full_like(xd, 7.0), new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, xd[:rows], pd, rd[:rows], residual=rd[:rows])
        sw.swin_block_gated_backward(h, xd[:rows], pd, yd[:rows], dx[:rows], grads)
        sw.swin_block_gated_sync_status(h)
    close(rd[:rows], ref, tol)
    assert torch.equal(rd[rows:].cpu(), r[rows:]) and (dx[rows:] == 7).all()


@pytest.mark.gpu
def test_empty_batch():
    C, F = 96, 256
    x, p, _, _ = make(0, C, F)
    xd, pd = dev(x), dev(p)
    grads = new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, xd, pd, xd.clone())
        sw.swin_block_gated_backward(h, xd, pd, xd.clone(), xd.clone(), grads)
        sw.swin_block_gated_sync_status(h)
    assert all(not v.any() for v in grads.values())


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40, 700])
def test_streams_and_captured_graphs_share_nothing(rows):
    C, F = 256, 640
    x, p, _, dy = make(rows, C, F, seed=5)
    x2, _, _, dy2 = make(rows, C, F, seed=6)
    pd = dev(p)
    a, b = (dev(x), dev(dy)), (dev(x2), dev(dy2))
    with gated(C, F) as h:
        def call(x, dy):
            out, dx, g = torch.empty_like(x), torch.empty_like(x), new_grads(p)
            sw.swin_block_gated_forward(h, x, pd, out)
            sw.swin_block_gated_backward(h, x, pd, dy, dx, g)
            return [out, dx] + [g[k] for k in sorted(g)]

        same = lambda o, w: all(torch.equal(i, j) for i, j in zip(o, w))  # noqa: E731
        want, want2 = call(*a), call(*b)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for k in range(6):
            with torch.cuda.stream(streams[k % 2]):
                got.append(call(*(a if k % 2 else b)))
        torch.cuda.synchronize()
        assert all(same(o, want if k % 2 else want2) for k, o in enumerate(got))
        graphs = []
        for t in (a, b):
            bufs = [v.clone() for v in t]
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                o = call(*bufs)
            graphs.append((gr, bufs, o))
        for v, t in zip(graphs[0][1], b):
            v.copy_(t)
        torch.cuda.synchronize()
        for (gr, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        eager = call(*a)
        torch.cuda.synchronize()
        sw.swin_block_gated_sync_status(h)
        assert same(graphs[0][2], want2) and same(graphs[1][2], want2) and same(eager, want)


@pytest.mark.gpu
def test_first_call_of_a_handle_captured():
    """A handle's first call may be the captured one."""
    rows, C, F = 300, 256, 384
    x, p, r, _ = make(rows, C, F, seed=11)
    ref, tol = forward_ref(x, p, r, "silu")
    xd, pd, rd, out = dev(x), dev(p), dev(r), torch.zeros(rows, C, dtype=BF, device=DEV)
    with gated(C, F) as h:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        for _ in range(2):
            gr.replay()
        sw.swin_block_gated_sync_status(h)
        close(out, ref, tol)
        del gr
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A hidden activation of more than 2^31 elements: the last rows, forward and
    backward."""
    rows, C, F = 33000, 136, 65536
    g = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)  # noqa: E731
    p = dict(Wg=n(F, C, std=C ** -0.5), Wu=n(F, C, std=C ** -0.5), Wd=n(C, F, std=F ** -0.5), bg=None, bu=None, bd=None)
    x, dy = n(rows, C), n(rows, C)
    out, dx, grads = torch.empty_like(x), torch.empty_like(x), new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, x, p, out)
        sw.swin_block_gated_backward(h, x, p, dy, dx, grads)
        sw.swin_block_gated_sync_status(h)
    host = {k: None if v is None else v.cpu() for k, v in p.items()}
    tail = slice(rows - 9, rows)
    ref, tol = forward_ref(x[tail].cpu(), host, None, "silu")
    close(out[tail], ref, tol)
    ref, tol = backward_ref(x[tail].cpu(), host, dy[tail].cpu(), "silu")
    close(dx[tail], ref["dx"], tol["dx"])
    assert all(torch.isfinite(v).all() for v in grads.values() if v is not None)


class env:
    def __init__(self, name):
        self.name = name

    def __enter__(self):
        os.environ[self.name] = "1"

    def __exit__(self, *exc):
        del os.environ[self.name]


@pytest.mark.gpu
def test_simulated_allocation_failure_then_a_normal_call():
    rows, C, F = 200, 192, 256
    x, p, _, dy = make(rows, C, F, seed=12)
    xd, pd, yd = dev(x), dev(p), dev(dy)
    out, grads = torch.full_like(xd, 5.0), new_grads(p)
    with gated(C, F) as h:
        with env("SWIN_WATTN_FAIL_ALLOC"):
            for call in (lambda: sw.swin_block_gated_forward(h, xd, pd, out),
                         lambda: sw.swin_block_gated_backward(h, xd, pd, yd, out, grads)):
                with pytest.raises(sw.SwinWAttnError) as ei:
                    call()
                assert ei.value.code == sw.ENOMEM
        torch.cuda.synchronize()
        assert (out == 5).all()
        sw.swin_block_gated_forward(h, xd, pd, out)
        sw.swin_block_gated_sync_status(h)
    ref, tol = forward_ref(x, p, None, "silu")
    close(out, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [(1, 96, 256), (70, 264, 520), (300, 1032, 2056), (700, 136, 264)])
def test_guard_bands_stay_intact_and_catch_an_overwrite(rows, C, F):
    x, p, r, dy = make(rows, C, F, seed=13)
    xd, pd, rd, yd = dev(x), dev(p), dev(r), dev(dy)
    out, dx, grads = torch.empty_like(xd), torch.empty_like(xd), new_grads(p)
    with env("SWIN_WATTN_DEBUG"), gated(C, F) as h:   # the bands are read back after each call
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        sw.swin_block_gated_backward(h, xd, pd, yd, dx, grads)
        for side in (0, 1):
            sw.swin_block_gated_test_corrupt_workspace(h, side)
            with pytest.raises(sw.SwinWAttnError) as ei:
                sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
            assert ei.value.code == sw.ECORRUPT


@pytest.mark.gpu
def test_bounded_waits_run_out():
    """Loads that never come: every role gives up, the status says so once, and
    the next call on the handle is right."""
    rows, C, F = 600, 256, 384
    x, p, r, _ = make(rows, C, F, seed=14)
    xd, pd, rd, out = dev(x), dev(p), dev(r), torch.empty(rows, C, dtype=BF, device=DEV)
    with gated(C, F) as h:
        sw.swin_block_gated_test_stall(h, xd, pd, 20000)
        with pytest.raises(sw.SwinWAttnError) as ei:
            sw.swin_block_gated_sync_status(h)
        assert ei.value.code == sw.ETIMEOUT
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        assert sw.swin_block_gated_sync_status(h) == sw.OK
    ref, tol = forward_ref(x, p, r, "silu")
    close(out, ref, tol)


@pytest.mark.gpu
@pytest.mark.parametrize("q8", [False, True])
def test_run_of_norm_and_gated_block(q8):
    """The second sub-layer of a pre-norm block, twice: (stream, branch) -> sum
    and its norm -> gated block added to the sum -> the next norm.  Against the
    same chain in float64 whose steps start from the library's own stored
    values, so that each step's bound applies."""
    rows, C, F = 333, 256, 640
    x, p, r, _ = make(rows, C, F, seed=7)
    gamma = (1 + 0.1 * torch.randn(C, generator=torch.Generator().manual_seed(1))).to(BF)
    xd, rd, pd, gd = dev(x), dev(r), dev(p), dev(gamma)
    s, n, out = torch.empty_like(xd), torch.empty_like(xd), torch.empty_like(xd)
    hn = sw.swin_block_rms_create(C, 1e-6)
    with gated(C, F) as h:
        if q8:
            codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.empty(rows, device=DEV)
            q = dict(pd)
            (q["Wg8"], q["sg"]), (q["Wu8"], q["su"]) = quantise(pd["Wg"]), quantise(pd["Wu"])
            sw.swin_block_rms_forward_q8(hn, xd, gd, codes, scales, residual=rd, out_sum=s)
            sw.swin_block_gated_forward_q8(h, codes, scales, q, out, residual=s)
            n = codes.double() * scales.double()[:, None]
            p = dict(p, Wg=q["Wg8"].double().cpu() * q["sg"].double().cpu()[:, None],
                     Wu=q["Wu8"].double().cpu() * q["su"].double().cpu()[:, None])
        else:
            sw.swin_block_rms_forward(hn, xd, gd, n, residual=rd, out_sum=s)
            sw.swin_block_gated_forward(h, n, pd, out, residual=s)
        sw.swin_block_gated_sync_status(h)
        assert torch.equal(s.cpu(), (x.float() + r.float()).to(BF))
        d = s.double().cpu()
        y = d / (d.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * gamma.double()
        step = (2.0 ** -4 * y.abs() + 2.0 ** -10 * y.abs().amax(-1, keepdim=True) / 448) if q8 else HALF * y.abs()
        assert ((n.double().cpu() - y).abs() <= step * 1.01).all()
        ref, tol = forward_ref(n.cpu(), p, s.cpu(), "silu")
        close(out, ref, tol)
        if not q8:   # the backward chain: dy -> (gated) dn -> (norm, the sum's own gradient added) ds
            dy = dev(make(rows, C, F, seed=8)[3])
            dn, ds, dgamma, grads = torch.empty_like(dy), torch.empty_like(dy), torch.empty(C, device=DEV), new_grads(p)
            sw.swin_block_gated_backward(h, n, pd, dy, dn, grads)
            sw.swin_block_rms_backward(hn, s, gd, dn, ds, dgamma, dsum=dy)
            sw.swin_block_gated_sync_status(h)
            ss = d.clone().requires_grad_()
            gg = gamma.double().requires_grad_()
            leaves = {k: v.double().requires_grad_() for k, v in p.items()}
            nn = ss / (ss.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * gg
            a = torch.nn.functional.silu(lin(nn, leaves["Wg"], leaves["bg"])) * lin(nn, leaves["Wu"], leaves["bu"])
            ((ss + lin(a, leaves["Wd"], leaves["bd"])) * dy.double().cpu()).sum().backward()
            # the chain's own roundings: n, dg / du, dn, each a relative 2^-8 at most, averaged over sums
            for got, want in [(ds, ss.grad), (dgamma, gg.grad)] + [(grads["d" + k], v.grad) for k, v in leaves.items()]:
                assert float((got.double().cpu() - want).norm() / want.norm()) <= 4 * HALF
    sw.swin_block_rms_destroy(hn)


@pytest.mark.gpu
def test_bias_gradients_of_infinite_units_leave_out_the_rows_behind():
    """A hidden unit whose u is infinite for every token: its dg is +inf in every
    row, and so is their sum; the zero rows that fill the last tile are not in
    it (there zero times infinity would be NaN)."""
    rows, C, F = 130, 64, 128
    x, p, _, dy = make(rows, C, F, seed=15)
    x, dy, p["Wd"] = x.abs() + 0.5, dy.abs() + 0.5, p["Wd"].abs() + 0.1
    p["Wg"] = p["Wg"].abs()   # act'(g) > 0 for every g of a positive row
    p["bg"].zero_()
    p["Wu"][5], p["bu"][9] = float("inf"), float("inf")
    p["Wu"][5] = p["Wu"][5].abs()
    dx, grads = torch.empty_like(dev(x)), new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_backward(h, dev(x), dev(p), dev(dy), dx, grads)
        sw.swin_block_gated_sync_status(h)
    dbg = grads["dbg"].cpu()
    assert dbg[5] == float("inf") and dbg[9] == float("inf")
    assert torch.isfinite(dbg[[i for i in range(F) if i not in (5, 9)]]).all()
    assert torch.isfinite(grads["dbu"]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [(5001, 144, 520), (5100, 144, 512), (19700, 144, 2056)])
def test_rounds_of_whole_tiles_and_a_last_one_in_parts(rows, C, F):
    """More tiles than CTA pairs, the last round thin: dealt out by halves and by
    quarters of tiles, or (the last product of the third) cut along K."""
    x, p, r, dy = make(rows, C, F, seed=16)
    ref, tol = forward_ref(x, p, r, "silu")
    xd, pd, rd, yd = dev(x), dev(p), dev(r), dev(dy)
    out, dx, grads = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan")), new_grads(p)
    x8, sx = quantise(x)
    q = dict(bg=p["bg"], bu=p["bu"], Wd=p["Wd"], bd=p["bd"])
    (q["Wg8"], q["sg"]), (q["Wu8"], q["su"]) = quantise(p["Wg"]), quantise(p["Wu"])
    exact = dict(p, Wg=q["Wg8"].double() * q["sg"].double()[:, None], Wu=q["Wu8"].double() * q["su"].double()[:, None])
    ref8, tol8 = forward_ref(x8.double() * sx.double()[:, None], exact, r, "silu")
    out8 = torch.full_like(xd, float("nan"))
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        sw.swin_block_gated_forward_q8(h, dev(x8), dev(sx), dev(q), out8, residual=rd)
        sw.swin_block_gated_backward(h, xd, pd, yd, dx, grads)
        sw.swin_block_gated_sync_status(h)
    close(out, ref, tol)
    close(out8, ref8, tol8)
    ref, tol = backward_ref(x, p, dy, "silu")
    for k, v in dict(grads, dx=dx).items():
        close(v, ref[k], tol[k])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [(300, 264, 8200), (300, 120, 8200), (9000, 136, 264), (20000, 136, 264)])
def test_products_cut_along_k(rows, C, F):
    """Few tiles of a long K: the forward's last product, dx (also in narrow
    tiles), the weight gradients by even ranges and by equal slices."""
    x, p, r, dy = make(rows, C, F, seed=17)
    xd, pd, rd, yd = dev(x), dev(p), dev(r), dev(dy)
    out, dx, grads = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan")), new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        if F > 8000 and C > 128:
            assert sw.swin_block_gated_last_launches(h) == 3   # (the third adds the partial tiles)
        sw.swin_block_gated_backward(h, xd, pd, yd, dx, grads)
        sw.swin_block_gated_sync_status(h)
    ref, tol = forward_ref(x, p, r, "silu")
    close(out, ref, tol)
    ref, tol = backward_ref(x, p, dy, "silu")
    for k, v in dict(grads, dx=dx).items():
        close(v, ref[k], tol[k])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", [(1300, 2048, 264), (2800, 1000, 136)])
def test_products_in_tiles_of_192_columns(rows, C, F):
    """Tiles of 256 columns for half of the CTA pairs and a few more: one round of
    narrower ones instead (the last product, dx, the weight gradients)."""
    x, p, r, dy = make(rows, C, F, seed=18)
    xd, pd, rd, yd = dev(x), dev(p), dev(r), dev(dy)
    out, dx, grads = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan")), new_grads(p)
    with gated(C, F, "gelu") as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        sw.swin_block_gated_backward(h, xd, pd, yd, dx, grads)
        sw.swin_block_gated_sync_status(h)
    ref, tol = forward_ref(x, p, r, "gelu")
    close(out, ref, tol)
    ref, tol = backward_ref(x, p, dy, "gelu")
    for k, v in dict(grads, dx=dx).items():
        close(v, ref[k], tol[k])


@pytest.mark.parametrize("stages", [5, 6])
def test_closing_waits_cover_every_release(stages):
    """Before a CTA ends, its loading warp waits for the last release of every
    stage that it filled, also where it filled fewer than there are.  Modelled on
    a barrier's rule: a wait for parity p passes once the phase of that parity
    has completed, and at once for parity 1 on a fresh barrier."""
    def passes(completed, parity):
        return (completed - 1) % 2 == parity   # (the phase that completed last; -1 before the first)

    for issued in range(0, 4 * stages + 2):
        uses = [len(range(s, issued, stages)) for s in range(stages)]   # releases of each stage's barrier
        seen = [sw.swin_block_gated_test_last_use(stages, issued, k) for k in range(min(stages, issued))]
        assert sorted(s for s, _ in seen) == [s for s in range(stages) if uses[s]]
        for s, parity in seen:
            assert passes(uses[s], parity), (issued, s)
            assert not passes(uses[s] - 1, parity), (issued, s)   # not before the last one
        with pytest.raises(sw.SwinWAttnError):
            sw.swin_block_gated_test_last_use(stages, issued, min(stages, issued))


# How the sizes of the tests above and below are divided (on 76 CTA pairs): per
# product (tiles, pairs, columns of a tile, half tiles, tiles cut along K, equal
# slices).
PLANS = {
    (5001, 144, 520): ((20, 40, 256, 40, 0, 0), (20, 40, 256, 40, 0, 0), (9, 76, 256, 0, 9, 0)),
    (19700, 144, 2056): ((77, 76, 256, 2, 0, 0), (77, 76, 256, 0, 1, 0), (27, 76, 256, 0, 27, 0)),
    (19700, 144, 4104): ((77, 76, 256, 0, 1, 0), (77, 76, 256, 0, 1, 0), (51, 76, 256, 0, 51, 0)),
    (300, 264, 8200): ((4, 76, 256, 0, 4, 0), (4, 76, 256, 0, 4, 0), (218, 76, 192, 0, 0, 0)),
    (300, 120, 8200): ((2, 64, 128, 0, 2, 0), (2, 76, 128, 0, 2, 0), (131, 76, 128, 0, 0, 0)),
    (20000, 136, 264): ((79, 76, 256, 6, 0, 0), (79, 76, 256, 6, 0, 0), (6, 72, 256, 0, 6, 1)),
    (1300, 2048, 264): ((66, 66, 192, 0, 0, 0), (66, 66, 192, 0, 0, 0), (60, 60, 192, 0, 0, 0)),
    (2800, 1000, 136): ((66, 66, 192, 0, 0, 0), (66, 66, 192, 0, 0, 0), (12, 24, 256, 24, 0, 0)),
}
# The one-kernel forward: (tiles, pairs, chunks, chunks held, all of them, one staging)
NARROW_PLANS = {
    (20000, 8, 136): (79, 76, 3, 3, 1, 0), (40000, 128, 136): (157, 76, 3, 3, 1, 1),
    (40000, 128, 200): (157, 76, 4, 3, 0, 1), (45001, 96, 256): (176, 76, 4, 4, 1, 1),
    (45000, 96, 320): (176, 76, 5, 4, 0, 1), (60001, 64, 64): (235, 76, 1, 1, 1, 0),
    (59000, 40, 328): (231, 76, 6, 6, 1, 0),
}


def test_the_tested_sizes_reach_the_plans_they_are_for():
    for (rows, C, F), want in PLANS.items():
        for which, w in zip((sw.BLOCK_GATED_PLAN_DOWN, sw.BLOCK_GATED_PLAN_DX, sw.BLOCK_GATED_PLAN_WEIGHTS), want):
            assert sw.swin_block_gated_test_plan(C, F, rows, which) == w, (rows, C, F, which)
    for (rows, C, F), w in NARROW_PLANS.items():
        assert sw.swin_block_gated_test_plan(C, F, rows, sw.BLOCK_GATED_PLAN_NARROW) == w, (rows, C, F)
    for bad in ((144, 64, 300, sw.BLOCK_GATED_PLAN_NARROW), (96, 64, 128, 0), (96, 12, 300, 0), (96, 64, 300, 4)):
        with pytest.raises(sw.SwinWAttnError):
            sw.swin_block_gated_test_plan(*bad)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F,launches", [(19700, 144, 2056, 2), (19700, 144, 4104, 3)])
def test_last_product_after_whole_rounds(rows, C, F, launches):
    """A whole round of tiles, then one tile as halves, or cut along K and joined
    by a third kernel, which adds bias and residual; from 16 and 8 bits, in place."""
    assert sw.swin_block_gated_test_plan(C, F, rows, sw.BLOCK_GATED_PLAN_DOWN) == PLANS[rows, C, F][0]
    x, p, r, _ = make(rows, C, F, seed=19)
    x8, sx = quantise(x)
    q = dict(bg=p["bg"], bu=p["bu"], Wd=p["Wd"], bd=p["bd"])
    (q["Wg8"], q["sg"]), (q["Wu8"], q["su"]) = quantise(p["Wg"]), quantise(p["Wu"])
    exact = dict(p, Wg=q["Wg8"].double() * q["sg"].double()[:, None], Wu=q["Wu8"].double() * q["su"].double()[:, None])
    xd, pd, rd = dev(x), dev(p), dev(r)
    out, out8, place = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan")), rd.clone()
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        assert sw.swin_block_gated_last_launches(h) == launches
        sw.swin_block_gated_forward(h, xd, pd, place, residual=place)
        sw.swin_block_gated_forward_q8(h, dev(x8), dev(sx), dev(q), out8, residual=rd)
        assert sw.swin_block_gated_last_launches(h) == launches
        sw.swin_block_gated_sync_status(h)
    for got, a, w in ((out, x, p), (out8, x8.double() * sx.double()[:, None], exact)):
        ref, tol = forward_ref(dev(a), dev(w), rd, "silu")
        close(got, ref.cpu(), tol.cpu())
    assert torch.equal(place, out)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", sorted(NARROW_PLANS))
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_narrow_tiles_with_biases_and_residual(rows, C, F, kind):
    """The one-kernel form with both over several tiles a pair: one staging or two,
    odd and even counts of chunks, weights that stay and that stream; in place."""
    assert sw.swin_block_gated_test_plan(C, F, rows, sw.BLOCK_GATED_PLAN_NARROW) == NARROW_PLANS[rows, C, F]
    x, p, r, _ = make(rows, C, F, seed=20)
    xd, pd, rd = dev(x), dev(p), dev(r)
    out, place = torch.full_like(xd, float("nan")), rd.clone()
    with gated(C, F, kind) as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        assert sw.swin_block_gated_last_launches(h) == 1
        sw.swin_block_gated_forward(h, xd, pd, place, residual=place)
        sw.swin_block_gated_sync_status(h)
    ref, tol = forward_ref(xd, pd, rd, kind)
    close(out, ref.cpu(), tol.cpu())
    assert torch.equal(place, out)


@pytest.mark.gpu
def test_sums_over_more_than_32_bits_of_hidden_elements():
    """The workspace of the offsets test (33000 x 65536 a matrix) with biases: rows at
    the beginning, where the 2^31st element lies and at the end of out and dx,
    and every gradient of hidden units at both ends and between, whose sums go
    over all rows."""
    rows, C, F = 33000, 136, 65536
    g = torch.Generator(device=DEV).manual_seed(6)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)  # noqa: E731
    p = dict(Wg=n(F, C, std=C ** -0.5), Wu=n(F, C, std=C ** -0.5), Wd=n(C, F, std=F ** -0.5), bg=n(F, std=0.3),
             bu=n(F, std=0.3), bd=n(C, std=0.3))
    x, dy = n(rows, C), n(rows, C)
    out, dx, grads = torch.empty_like(x), torch.empty_like(x), new_grads(p)
    with gated(C, F) as h:
        sw.swin_block_gated_forward(h, x, p, out)
        sw.swin_block_gated_backward(h, x, p, dy, dx, grads)
        sw.swin_block_gated_sync_status(h)
    some = [0, 1, 255, 256, 20000, 32766, 32767, 32768, 32769, 32999]
    ref, tol = forward_ref(x[some], p, None, "silu")
    close(out[some], ref.cpu(), tol.cpu())
    ref, tol = backward_ref(x[some], p, dy[some], "silu")
    close(dx[some], ref["dx"].cpu(), tol["dx"].cpu())
    units = list(range(8)) + list(range(127, 129)) + list(range(32760, 32776)) + list(range(50000, 50007))
    units += list(range(F - 64, F))
    part = dict(Wg=p["Wg"][units], Wu=p["Wu"][units], Wd=p["Wd"][:, units], bg=p["bg"][units], bu=p["bu"][units],
                bd=p["bd"])
    ref, tol = backward_ref(x, part, dy, "silu")
    got = dict(dWg=grads["dWg"][units], dWu=grads["dWu"][units], dWd=grads["dWd"][:, units], dbg=grads["dbg"][units],
               dbu=grads["dbu"][units], dbd=grads["dbd"])
    for k, v in got.items():
        close(v, ref[k].cpu(), tol[k].cpu())


@pytest.mark.gpu
def test_two_host_threads_compute_what_one_does():
    """A handle a thread, on streams of their own, at once: every result is the one
    that the same call gives alone."""
    import threading
    cases = [(1, 256, 640), (700, 256, 640), (300, 96, 256), (1000, 512, 1368)]
    wrong = []

    def call(h, x, p, dy):
        out, dx, g = torch.empty_like(x), torch.empty_like(x), new_grads(p)
        sw.swin_block_gated_forward(h, x, p, out)
        sw.swin_block_gated_backward(h, x, p, dy, dx, g)
        return [out, dx] + [g[k] for k in sorted(g)]

    data = []
    for rows, C, F in cases:
        x, p, _, dy = make(rows, C, F, seed=21)
        x, p, dy = dev(x), dev(p), dev(dy)
        with gated(C, F) as h:
            want = call(h, x, p, dy)
            sw.swin_block_gated_sync_status(h)
        data.append((C, F, x, p, dy, want))
    torch.cuda.synchronize()

    def work(C, F, x, p, dy, want):
        try:
            stream = torch.cuda.Stream()
            with gated(C, F) as h, torch.cuda.stream(stream):
                for _ in range(30):
                    got = call(h, x, p, dy)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append((C, F))
                sw.swin_block_gated_sync_status(h)
        except Exception as e:
            wrong.append((C, F, e))

    threads = [threading.Thread(target=work, args=a) for a in data]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


TWO_KERNEL_NARROW = [(129, 128, 4096), (263, 40, 992), (700, 24, 20000), (1180, 8, 6152), (3000, 8, 4096),
                     (20000, 128, 4096)]


def test_few_narrow_tiles_of_a_long_hidden_width_are_spread_over_the_pairs():
    """The one kernel walks all of F in the pair of a row tile: with few tiles (or a
    last round of few) two kernels are up to nine times faster."""
    for rows, C, F in TWO_KERNEL_NARROW:
        with pytest.raises(sw.SwinWAttnError):
            sw.swin_block_gated_test_plan(C, F, rows, sw.BLOCK_GATED_PLAN_NARROW)
    for rows, C, F in ((129, 128, 512), (1000, 128, 576), (30000, 64, 4096), (75936, 104, 3896), (200704, 128, 2048)):
        sw.swin_block_gated_test_plan(C, F, rows, sw.BLOCK_GATED_PLAN_NARROW)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,F", TWO_KERNEL_NARROW)
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_narrow_tokens_by_two_kernels(rows, C, F, kind):
    """With biases and residual, without either, and in place."""
    x, p, r, _ = make(rows, C, F, seed=22)
    xd, pd, rd = dev(x), dev(p), dev(r)
    bare = {k: None if k.startswith("b") else v for k, v in pd.items()}
    out, plain, place = torch.full_like(xd, float("nan")), torch.full_like(xd, float("nan")), rd.clone()
    with gated(C, F, kind) as h:
        sw.swin_block_gated_forward(h, xd, pd, out, residual=rd)
        assert sw.swin_block_gated_last_launches(h) in (2, 3)
        sw.swin_block_gated_forward(h, xd, bare, plain)
        sw.swin_block_gated_forward(h, xd, pd, place, residual=place)
        sw.swin_block_gated_sync_status(h)
    for got, w, res in ((out, pd, rd), (plain, bare, None)):
        ref, tol = forward_ref(xd, w, res, kind)
        close(got, ref.cpu(), tol.cpu())
    assert torch.equal(place, out)
