"""The linear operator (include/swin_linear.h).

CPU (not gpu): refusals, the division of products, and the gradient formulas
against autograd in float64 and against differences.  GPU: forward (bf16,
8-bit) and backward against the formulas in float64, at sizes on each side of
the kernels' tiles and plans (one row, tiles that end inside, halves, K cut by
ranges and by slices), biases, residuals, kept values and gradients present or
not, in place, on two streams, captured and replayed, and the runs a block makes
of it: norm -> GELU layer -> layer with the residual, and the merging step.

Tolerances: a stored bf16 value is off by at most HALF = 2^-8 of itself.  A sum
of K products in fp32 takes K / 16 additions one after the other, each off by at
most 2^-23 of the largest partial sum, S = sum |x w| + |b| at most: E = (K / 8 +
16) 2^-23 S (twice that: the products of one step are added too).  The
activation's slope is at most 1.13, its own error 2^-17 (1 + |z|) (an erf good to
5.5e-7, the approximate exponential and reciprocal).  dz is rounded to bf16: an
error of HALF |dz| goes through the products that read it.  These are worst
cases, so the relative error in the 2-norm is held too: a rounding of at most
2^-8 each.
"""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from vision_transformer_shifted_gb300 import binding as sw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF = 2.0 ** -8
ACTS = {"none": sw.BLOCK_LINEAR_NONE, "silu": sw.BLOCK_LINEAR_SILU, "gelu": sw.BLOCK_LINEAR_GELU}


def act(z, kind):
    """act(z) and act'(z)."""
    if kind == "none":
        return z, torch.ones_like(z)
    if kind == "silu":
        p = torch.sigmoid(z)
        return z * p, p * (1 + z * (1 - p))
    phi = torch.special.ndtr(z)
    return z * phi, phi + z * torch.exp(-z * z / 2) / (2 * torch.pi) ** 0.5


def chain(k):
    return (k / 8 + 16) * 2.0 ** -23


def forward_ref(x, w, b, residual, kind):
    """z, out and the bounds on their errors (float64)."""
    x, w = x.double(), w.double()
    z, s = x @ w.t(), x.abs() @ w.abs().t()
    if b is not None:
        z, s = z + b.double(), s + b.double().abs()
    e = chain(x.shape[1]) * s
    out = act(z, kind)[0]
    eo = 1.13 * e + (0 if kind == "none" else 2.0 ** -17 * (1 + z.abs()))
    if residual is not None:
        out = out + residual.double()
    return z, out, HALF * 1.01 * z.abs() + e, HALF * 1.01 * out.abs() + 1.01 * eo


def backward_ref(x, w, z, dy, kind):
    """Gradients and the bounds on their errors (float64)."""
    x, w, dy = x.double(), w.double(), dy.double()
    dz, e = dy, torch.zeros_like(dy)
    if kind != "none":
        dz = dy * act(z.double(), kind)[1]
        e = 2.0 ** -17 * (1 + z.double().abs()) * dy.abs()
    rounded = e + (0 if kind == "none" else HALF * dz.abs())
    ref = dict(dx=dz @ w, dW=dz.t() @ x, db=dz.sum(0))
    err = dict(dx=rounded @ w.abs() + chain(w.shape[0]) * (dz.abs() @ w.abs()),
               dW=rounded.t() @ x.abs() + chain(x.shape[0]) * (dz.abs().t() @ x.abs()),
               db=e.sum(0) + 2.0 ** -17 * dz.abs().sum(0))
    return ref, {k: HALF * 1.01 * ref[k].abs() + err[k] for k in ref}


def close(got, ref, tol, rel=HALF):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= tol + 1e-30).all(), float((err - tol).max())
    if ref.numel() >= 64:   # (a norm of many roundings)
        assert float(err.norm() / ref.norm()) <= rel


def make(rows, C, N, bias=True, residual=True, seed=0):
    """x, W, b, residual, dy."""
    g = torch.Generator().manual_seed(seed * 7919 + rows * 31 + C * 17 + N)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    return (n(rows, C), n(N, C, std=C ** -0.5), n(N, std=0.3) if bias else None, n(rows, N) if residual else None,
            n(rows, N))


def dev(*ts):
    out = [None if t is None else t.to(DEV) for t in ts]
    return out if len(out) > 1 else out[0]


def nans(*shape):
    return torch.full(shape, float("nan"), dtype=BF, device=DEV)


def quantise(w):
    s = w.float().abs().amax(-1).clamp_min(1e-30) / 448
    return (w.float() / s[:, None]).to(E4M3), s


def stored_z(x, w, b):
    """z as a forward keeps it."""
    return (x.double() @ w.double().t() + (0 if b is None else b.double())).to(BF)


class linear:
    def __init__(self, C, N, kind="none"):
        self.args = C, N, ACTS[kind]

    def __enter__(self):
        self.h = sw.swin_block_linear_create(*self.args)
        return self.h

    def __exit__(self, *exc):
        sw.swin_block_linear_destroy(self.h)


class env:
    def __init__(self, name):
        self.name = name

    def __enter__(self):
        os.environ[self.name] = "1"

    def __exit__(self, *exc):
        del os.environ[self.name]


# ---- CPU ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_gradient_formulas(kind):
    g = torch.Generator().manual_seed(11)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    p = dict(x=n(5, 8), W=n(16, 8) * 0.4, b=n(16))
    dy = n(5, 16)

    def loss(p):
        z = p["x"] @ p["W"].t() + p["b"]
        f = {"none": lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[kind]
        return (f(z) * dy).sum()

    ref, _ = backward_ref(p["x"], p["W"], p["x"] @ p["W"].t() + p["b"], dy, kind)
    leaves = {k: v.clone().requires_grad_() for k, v in p.items()}
    loss(leaves).backward()
    for k, t in leaves.items():
        assert torch.allclose(ref["d" + k], t.grad, rtol=1e-12, atol=1e-12), k
        for i in (0, 3, t.numel() - 1):   # and three entries each against a central difference
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = 1e-5
            diff = float(loss(dict(p, **{k: p[k] + e.view(t.shape)})) - loss(dict(p, **{k: p[k] - e.view(t.shape)}))) / 2e-5
            assert abs(diff - float(ref["d" + k].reshape(-1)[i])) < 1e-6 * (1 + abs(diff)), k


@pytest.mark.parametrize("C,N,kind", [(0, 64, 0), (12, 64, 0), (64, 0, 0), (64, 12, 0), (-8, 64, 0), (65544, 64, 0),
                                      (64, 65544, 0), (64, 64, 3), (64, 64, -1)])
def test_create_refuses(C, N, kind):
    h = ctypes.c_void_p(1)
    assert sw.load().swin_block_linear_create(ctypes.byref(h), C, N, kind) == sw.EINVAL
    assert h.value is None
    assert sw.load().swin_block_linear_create(None, 64, 64, 0) == sw.EINVAL


P = 1 << 24   # addresses that no refused call reads
STEP = 1 << 16


def _addresses(names):
    return {n: P + i * STEP for i, n in enumerate(names)}


def test_forward_refuses():
    lib = sw.load()
    ok = _addresses(["W", "b", "x", "residual", "z", "out", "sx", "sw"])

    def call(q8, rows=4, C=64, kind="gelu", **kw):
        a = {**ok, **kw}
        with linear(C, 64, kind) as h:
            h = a.get("h", h)
            if q8:
                return lib.swin_block_linear_forward_q8(h, a["x"], a["sx"], rows, a["W"], a["sw"], a["b"], a["residual"],
                                                        a["out"], None)
            return lib.swin_block_linear_forward(h, a["x"], rows, a["W"], a["b"], a["residual"], a["z"], a["out"], None)

    both = [dict(h=None), dict(rows=-1), dict(rows=(1 << 31) - 1)]
    both += [{n: None} for n in ("W", "x", "out")]
    both += [{n: ok[n] + 8} for n in ("W", "b", "x", "residual", "out")]
    both += [dict(out=ok[n]) for n in ("W", "b", "x")]
    both += [dict(out=ok["residual"] + 16)]
    for bad in both:
        assert call(False, **bad) == sw.EINVAL, bad
        assert call(True, **bad) == sw.EINVAL, bad
    for bad in [dict(z=ok["z"] + 2), dict(kind="none")] + [dict(z=ok[n]) for n in ("W", "b", "x", "residual", "out")]:
        assert call(False, **bad) == sw.EINVAL, bad
    for bad in [{n: None} for n in ("sx", "sw")] + [{n: ok[n] + 4} for n in ("sx", "sw")] + [
            dict(out=ok[n]) for n in ("sx", "sw")]:
        assert call(True, **bad) == sw.EINVAL, bad
    assert call(False, rows=0) == sw.OK and call(True, rows=0) == sw.OK
    assert call(True, C=72) == sw.EUNSUPPORTED
    assert lib.swin_block_linear_destroy(None) == sw.OK
    assert lib.swin_block_linear_last_launches(None) == 0
    assert lib.swin_block_linear_sync_status(None, None) == sw.EINVAL


def test_backward_refuses():
    lib = sw.load()
    ins, outs = ["x", "W", "z", "dy"], ["dx", "dW", "db"]
    ok = _addresses(ins + outs)

    def call(rows=4, kind="silu", **kw):
        a = {**ok, **kw}
        with linear(64, 64, kind) as h:
            return lib.swin_block_linear_backward(a.get("h", h), a["x"], rows, a["W"], a["z"], a["dy"], a["dx"], a["dW"],
                                                  a["db"], None)

    bad = [dict(h=None), dict(rows=-1), dict(rows=(1 << 31) - 1), dict(kind="none"), dict(dx=None, dW=None),
           dict(dx=None, dW=None, db=None), dict(dW=None)]
    bad += [{n: None} for n in ins]
    bad += [{n: ok[n] + 2} for n in ok]
    bad += [{o: ok[i]} for o in outs for i in ins]
    bad += [dict(dx=ok["dW"]), dict(db=ok["dx"]), dict(db=ok["dW"] + 16)]
    for b in bad:
        assert call(**b) == sw.EINVAL, b


def test_binding_refuses_other_types_shapes_and_devices():
    x, w, b, r, dy = make(4, 64, 128)
    out = torch.empty(4, 128, dtype=BF)
    with linear(64, 128, "gelu") as h:
        for kw in (dict(x=x.float()), dict(x=dy), dict(w=w.float()), dict(w=w.t().contiguous()), dict(b=b[:64]),
                   dict(out=x.clone()), dict(residual=r[:2]), dict(z=out.float()), {}):   # (the last: on the CPU)
            a = {**dict(x=x, w=w, b=b, out=out, residual=r, z=out.clone()), **kw}
            with pytest.raises(ValueError):
                sw.swin_block_linear_forward(h, a["x"], a["w"], a["b"], a["out"], residual=a["residual"], z=a["z"])
        with pytest.raises(ValueError):
            sw.swin_block_linear_backward(h, x, w, dy, x.clone(), w.clone(), b.clone(), z=dy.clone())
        with pytest.raises(ValueError):
            sw.swin_block_linear_forward_q8(h, x, torch.ones(4), w, torch.ones(128), b, out)


FWD, Q8, DX, DW = (sw.BLOCK_LINEAR_PLAN_FORWARD, sw.BLOCK_LINEAR_PLAN_FORWARD_Q8, sw.BLOCK_LINEAR_PLAN_DX,
                   sw.BLOCK_LINEAR_PLAN_WEIGHT)


def test_plans_of_the_tested_sizes():
    """Tiles of 256, 192 and 128 columns, half tiles alone and behind whole rounds,
    K cut by even ranges and by equal slices: what LARGE and SHAPES reach on 152
    SMs."""
    for args, want in [   # columns of a tile, half tiles, cut along K, into equal slices
            ((328, 136, 129, FWD), (256, 1, 0, 0)), ((2048, 2056, 1300, FWD), (192, 0, 0, 0)),
            ((8192, 1032, 1000, FWD), (256, 0, 1, 0)),
            ((512, 2048, 2500, Q8), (256, 1, 0, 0)), ((264, 336, 20000, FWD), (192, 0, 0, 0)),
            ((136, 6792, 4067, DX), (256, 0, 1, 0)),
            ((144, 520, 5001, DW), (256, 0, 1, 0)), ((96, 384, 20000, DW), (128, 0, 1, 0)),
            ((520, 1032, 6000, DW), (256, 0, 1, 1))]:
        tiles, pairs, columns, halves, cut, equal = sw.swin_block_linear_test_plan(*args)
        assert pairs and (columns, halves > 0, cut > 0, equal) == want, args
    for args in ((4096, 120, 700, FWD), (8208, 264, 300, FWD), (2968, 400, 385, FWD), (4096, 1024, 300, Q8),
                 (264, 8200, 300, DX), (120, 8200, 300, DX)):
        assert sw.swin_block_linear_test_plan(*args)[1] == 0, args   # (the few-row kernel, in chunks of rows)


def test_plans_of_the_weight_gradient_through_an_activation():
    """Tiles of one and of two columns' MMAs, several across, one slice and many, and
    sizes where dz is formed apart: what the tested sizes reach on 152 SMs."""
    plan = lambda *a: sw.swin_block_linear_test_plan(*a, sw.BLOCK_LINEAR_PLAN_ACT_WEIGHT)  # noqa: E731
    for args, want in [   # columns of a tile, tiles across, slices
            ((96, 384, 20000), (96, 1, 35)), ((512, 2048, 2500), (512, 1, 8)), ((768, 768, 3000), (384, 2, 12)),
            ((1032, 1000, 4000), (352, 3, 6)), ((8, 136, 4000), (64, 1, 63)), ((24, 10008, 10000), (64, 1, 1)),
            ((2048, 264, 5000), (512, 4, 9))]:
        tiles, pairs, columns, across, slices, chosen = plan(*args)
        assert chosen and (columns, across, slices) == want and pairs == tiles * slices, args
    for args in ((512, 1368, 1), (4096, 120, 700), (1032, 2056, 300), (136, 65536, 33000), (96, 128, 128)):
        assert not plan(*args)[5], args


GRADS = sw.BLOCK_LINEAR_GRAD_DX, sw.BLOCK_LINEAR_GRAD_DW, sw.BLOCK_LINEAR_GRAD_DB
ALL = sum(GRADS)


@pytest.mark.parametrize("kind", ["none", "gelu"])
@pytest.mark.parametrize("which", [ALL, 3, 1, 2, 6])   # (db never without dW)
def test_whoever_adds_the_rows_of_db_has_them(kind, which):
    """One kernel, and one only, finishes db, and where it adds partial rows the
    workspace holds them: dW's epilogue to the end (rows of dy, or held rows of dz's
    sums), dx's epilogue, or a launch of its own."""
    widths = [8, 64, 96, 264, 512, 1000, 1032, 2048, 4096, 7424, 8192, 11008, 12288, 16384, 20480, 32768, 65536]
    lengths = [*range(1, 600, 13), 128, 129, 200, 256, 257, 1000, 2000, 5000, 20000, 70000]
    for C in widths:
        for N in widths:
            for rows in lengths:
                p = sw.swin_block_linear_test_backward_plan(C, N, rows, ACTS[kind], which)
                at = (rows, C, N, p)
                db = which & GRADS[2]
                assert not (p["direct"] or p["dx_adds"]) or db, at
                assert not (p["direct"] and p["dx_adds"]), at
                assert not p["dx_adds"] or (p["side"] and p["held"] and p["slices"] <= 512), at
                assert not p["direct"] or (p["slices"] if kind != "none" else rows) <= 256, at
                assert not db or p["held"] or (p["direct"] and kind == "none"), at
                assert not p["side"] or (which & 3 == 3 and not p["few"] and not p["dx_cut"]
                                         and (p["through"] or p["dw_cut"] or p["dx_adds"])), at


def test_every_way_of_finishing_a_backward_is_tested():
    widths = [8, 64, 264, 512, 1000, 1032, 2048, 4096, 7424, 8192, 12288, 16384, 32768, 65536]
    lengths = [1, 40, 128, 129, 200, 256, 257, 300, 500, 1000, 1300, 2000, 5000, 20000, 70000]

    def way(rows, C, N, kind):
        p = sw.swin_block_linear_test_backward_plan(C, N, rows, ACTS[kind], ALL)
        return kind, *(k for k, v in p.items() if v and k not in ("slices", "held"))

    tested = {way(*s) for s in FINISHING}
    tested |= {way(*s, kind) for s in SHAPES + LARGE for kind in ("none", "gelu")}
    for C in widths:
        for N in widths:
            for rows in lengths:
                for kind in ("none", "gelu"):
                    assert way(rows, C, N, kind) in tested, (rows, C, N, way(rows, C, N, kind))


def test_backward_plan_refuses():
    for a in ((0, 8, 300, 0, 7), (8, 12, 300, 0, 7), (8, 8, 0, 0, 7), (8, 8, 300, 0, 0), (8, 8, 300, 0, 4), (8, 8, 300, 0, 5),
              (8, 8, 300, 0, 8)):
        with pytest.raises(sw.SwinWAttnError):
            sw.swin_block_linear_test_backward_plan(*a)


def test_clusters_that_find_room_are_a_devices_own():
    """What one device says is not taken for another (these two are no machine's)."""
    of = sw.swin_block_linear_test_clusters_of
    assert of(62, 8, False, 0) == 0   # (no answer is not kept)
    assert of(62, 8, False, 36) == 36 and of(63, 8, False, 20) == 20
    assert of(62, 8, False, 5) == 36 and of(63, 8, False, 5) == 20
    assert of(62, 8, True, 18) == 18 and of(62, 16, False, 7) == 7
    assert of(64, 8, False, 11) == 11 and of(64, 8, False, 12) == 12   # (past the table: asked each time)
    assert of(0, 17, False, 1) == of(0, 0, False, 1) == sw.EINVAL


def test_plan_refuses():
    for a in ((0, 8, 300, 0), (8, 12, 300, 0), (8, 8, 0, 0), (8, 8, 300, 5)):
        with pytest.raises(sw.SwinWAttnError):
            sw.swin_block_linear_test_plan(*a)


# ---- GPU ---------------------------------------------------------------------------

SHAPES = [   # rows, C, N
    (1, 8, 8), (1, 96, 384), (1, 512, 1368), (1, 8208, 40), (1, 1040, 6152), (2, 64, 64), (5, 136, 120), (17, 128, 264), (24, 1024, 2048),
    (64, 256, 640), (127, 192, 512), (128, 96, 128), (129, 328, 136), (256, 512, 512), (300, 1032, 2056),
    (515, 128, 384), (385, 2968, 400), (1000, 64, 1024), (3001, 96, 384), (2048, 768, 1024), (700, 4096, 120), (300, 8208, 264),
    (40, 2048, 4864), (100, 520, 720)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", SHAPES)
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_forward(rows, C, N, kind):
    x, w, b, r, _ = make(rows, C, N)
    xd, wd, bd, rd = dev(x, w, b, r)
    with linear(C, N, kind) as h:
        for bias in (bd, None):
            for res in (rd, None):
                z, out, ez, eo = forward_ref(x, w, None if bias is None else b, None if res is None else r, kind)
                got = nans(rows, N)
                sw.swin_block_linear_forward(h, xd, wd, bias, got, residual=res)
                sw.swin_block_linear_sync_status(h)
                close(got, out, eo)
                if kind != "none":
                    kept, again = nans(rows, N), nans(rows, N)
                    sw.swin_block_linear_forward(h, xd, wd, bias, again, residual=res, z=kept)
                    sw.swin_block_linear_sync_status(h)
                    close(kept, z, ez)
                    assert torch.equal(got, again)   # (kept or not)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [s for s in SHAPES if s[1] % 16 == 0])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_forward_q8(rows, C, N, kind):
    x, w, b, r, _ = make(rows, C, N, seed=1)
    (x8, sx), (w8, sc) = quantise(x), quantise(w)
    exact = x8.double() * sx.double()[:, None], w8.double() * sc.double()[:, None]
    with linear(C, N, kind) as h:
        for bias in (b, None):
            for res in (r, None):
                _, out, _, eo = forward_ref(*exact, bias, res, kind)
                got = nans(rows, N)
                sw.swin_block_linear_forward_q8(h, *dev(x8, sx, w8, sc, bias), got, residual=None if res is None else dev(res))
                sw.swin_block_linear_sync_status(h)
                close(got, out, eo)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", SHAPES + [(300, 264, 8200), (300, 120, 8200)])
@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_backward(rows, C, N, kind):
    x, w, b, _, dy = make(rows, C, N, seed=2)
    z = None if kind == "none" else stored_z(x, w, b)
    ref, tol = backward_ref(x, w, z, dy, kind)
    xd, wd, zd, yd = dev(x, w, z, dy)
    rel = 2 * HALF
    with linear(C, N, kind) as h:
        got = [dict(dx=nans(rows, C), dW=nans(N, C), db=nans(N)) for _ in range(2)]
        for g in got:
            sw.swin_block_linear_backward(h, xd, wd, yd, g["dx"], g["dW"], g["db"], z=zd)
        only = dict(dx=nans(rows, C), dW=nans(N, C))
        sw.swin_block_linear_backward(h, xd, wd, yd, only["dx"], None, z=zd)   # frozen parameters
        sw.swin_block_linear_backward(h, xd, wd, yd, None, only["dW"], z=zd)   # the first layer, no bias
        sw.swin_block_linear_sync_status(h)
    for k in ref:
        close(got[0][k], ref[k], tol[k], rel)
        assert torch.equal(got[0][k], got[1][k]), k   # a fixed order of summation
    for k in only:
        assert torch.equal(only[k], got[0][k]), k


LARGE = [   # rows, C, N: more tiles than CTA pairs, thin last rounds, long K
    (2500, 512, 2048), (5001, 144, 520), (1300, 2048, 2056), (20000, 264, 336), (20000, 96, 384), (6000, 520, 1032),
    (9000, 384, 96), (3000, 768, 768), (4000, 1032, 1000), (4000, 8, 136), (10000, 24, 10008), (5000, 2048, 264),
    (1000, 8192, 1032), (4067, 136, 6792), (300, 4096, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", LARGE)
def test_rounds_of_tiles_and_products_cut_along_k(rows, C, N):
    x, w, b, r, dy = make(rows, C, N, seed=16)
    xd, wd, bd, rd, yd = dev(x, w, b, r, dy)
    z, out, ez, eo = forward_ref(xd, wd, bd, rd, "gelu")
    got, kept, out8 = nans(rows, N), nans(rows, N), nans(rows, N)
    g = dict(dx=nans(rows, C), dW=nans(N, C), db=nans(N))
    with linear(C, N, "gelu") as h:
        sw.swin_block_linear_forward(h, xd, wd, bd, got, residual=rd, z=kept)
        plain = nans(rows, N)
        sw.swin_block_linear_forward(h, xd, wd, bd, plain, residual=rd)
        sw.swin_block_linear_backward(h, xd, wd, yd, g["dx"], g["dW"], g["db"], z=kept)
        if C % 16 == 0:
            (x8, sx), (w8, sc) = quantise(xd), quantise(wd)
            sw.swin_block_linear_forward_q8(h, x8, sx, w8, sc, bd, out8, residual=rd)
        sw.swin_block_linear_sync_status(h)
    close(got, out.cpu(), eo.cpu())
    close(kept, z.cpu(), ez.cpu())
    assert torch.equal(plain, got)
    if C % 16 == 0:
        _, ref, _, tol = forward_ref(x8.double() * sx.double()[:, None], w8.double() * sc.double()[:, None], bd, rd, "gelu")
        close(out8, ref.cpu(), tol.cpu())
    ref, tol = backward_ref(xd, wd, kept, yd, "gelu")
    for k in ref:
        close(g[k], ref[k].cpu(), tol[k].cpu(), 2 * HALF)


FINISHING = [   # rows, C, N, kind: who finishes dx, dW and db, as SHAPES and LARGE do not have it
    (200, 8192, 2048, "none"), (256, 12288, 4096, "none"), (129, 65536, 512, "none"), (160, 7424, 8, "none"),
    (257, 8, 32768, "none"), (129, 8, 32768, "none"), (257, 8, 4096, "none"), (3000, 8, 2048, "none"),
    (5000, 1000, 7424, "none"), (20000, 64, 8, "none"), (1300, 64, 1032, "gelu"), (1300, 64, 2048, "gelu"),
    (70000, 64, 64, "gelu"), (2000, 64, 2048, "gelu"), (5000, 1000, 7424, "gelu"), (1300, 64, 4096, "gelu"),
    (20000, 64, 8, "gelu"), (129, 8, 32768, "gelu"), (131, 7424, 8, "gelu"), (200, 8192, 2048, "gelu")]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N,kind", FINISHING + [(*s, "none") for s in LARGE])
def test_who_finishes_what_of_a_backward(rows, C, N, kind):
    x, w, b, _, dy = make(rows, C, N, seed=33)
    xd, wd, yd, bd = dev(x, w, dy, b)
    z = None if kind == "none" else stored_z(xd, wd, bd)
    ref, tol = backward_ref(xd, wd, z, yd, kind)
    got = [dict(dx=nans(rows, C), dW=nans(N, C), db=nans(N)) for _ in range(3)]
    with linear(C, N, kind) as h:
        for g in got[:2]:
            sw.swin_block_linear_backward(h, xd, wd, yd, g["dx"], g["dW"], g["db"], z=z)
        sw.swin_block_linear_backward(h, xd, wd, yd, got[2]["dx"], got[2]["dW"], z=z)   # without db
        sw.swin_block_linear_sync_status(h)
    for k in ref:
        assert torch.equal(got[0][k], got[1][k]), k
        for g in got[::2]:
            if g is got[0] or k != "db":
                close(g[k], ref[k].cpu(), tol[k].cpu(), 2 * HALF)
    assert got[2]["db"].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 300])
def test_nan_and_infinity_stay_in_their_rows_and_columns(rows):
    C, N = 264, 328
    x, w, b, r, dy = make(rows, C, N, seed=3)
    x[7, 3], w[11, 5], b[13] = float("nan"), float("inf"), float("inf")
    r[9, 20] = float("nan")
    good_rows, good = [i for i in range(rows) if i not in (7,)], [i for i in range(N) if i not in (11, 13)]
    _, out, _, eo = forward_ref(x[good_rows], w[good], b[good], r[good_rows][:, good], "silu")
    got, kept = nans(rows, N), nans(rows, N)
    with linear(C, N, "silu") as h:
        sw.swin_block_linear_forward(h, *dev(x, w, b), got, residual=dev(r), z=kept)
        sw.swin_block_linear_sync_status(h)
    got = got.cpu()
    assert got[7].isnan().all() and got[9, 20].isnan() and (kept[good_rows][:, 13] == float("inf")).all()
    assert not got[:, 11].isfinite().any()
    part = got[good_rows][:, good]
    at = torch.zeros_like(part, dtype=torch.bool)
    at[good_rows.index(9), good.index(20)] = True
    assert part[~at].isfinite().all()
    err = (part.double() - out).abs()
    assert (err[~at] <= eo[~at]).all()


@pytest.mark.gpu
def test_one_row_with_nan_and_infinity():
    """Single tokens have a kernel of their own: what is not finite stays in its
    channel, or, in x, reaches all; e4m3 NaN codes too."""
    C, N = 528, 136
    x, w, b, r, _ = make(1, C, N, seed=20)
    w[11, 5], b[13], r[0, 20] = float("inf"), float("-inf"), float("nan")
    good = [i for i in range(N) if i not in (11, 13, 20)]
    _, out, _, eo = forward_ref(x, w[good], b[good], r[:, good], "gelu")
    got, kept = nans(1, N), nans(1, N)
    (x8, sx), (w8, sc) = quantise(x), quantise(make(1, C, N, seed=20)[1])
    w8 = w8.view(torch.uint8)
    w8[17, 500] = 0x7f   # NaN
    w8 = w8.view(E4M3)
    got8 = nans(1, N)
    with linear(C, N, "gelu") as h:
        sw.swin_block_linear_forward(h, *dev(x, w, b), got, residual=dev(r), z=kept)
        sw.swin_block_linear_forward_q8(h, *dev(x8, sx, w8, sc), None, got8)
        x[0, 500] = float("nan")
        bad = nans(1, N)
        sw.swin_block_linear_forward(h, *dev(x, w, b), bad)
        sw.swin_block_linear_sync_status(h)
    close(got[:, good], out, eo)
    assert not got[0, [11]].isfinite().any() and got[0, 20].isnan() and kept[0, 13] == float("-inf")
    assert bad.isnan().all()
    assert got8[0, 17].isnan() and got8.isnan().sum() == 1


FAR = [1e30, -1e30, 3e38, -3e38, 2e19, -2e19, 100.0, -100.0]   # act is z or 0 there, act' 1 or 0


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(1, 64, 264), (40, 64, 264), (300, 64, 264), (385, 2968, 400)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_activation_far_from_zero(rows, C, N, kind):
    x, w, _, r, _ = make(rows, C, N, seed=23)
    far = torch.tensor(FAR).repeat(N // 8).to(BF)
    (x8, sx), (w8, sc) = quantise(x), quantise(torch.zeros_like(w))
    want = far.clamp_min(0).expand(rows, N)
    want = want, (want.float() + r.float()).to(BF)
    got, z, got8 = nans(rows, N), nans(rows, N), nans(rows, N)
    with linear(C, N, kind) as h:
        for res, ref in zip((None, dev(r)), want):
            sw.swin_block_linear_forward(h, dev(x), torch.zeros_like(w, device=DEV), dev(far), got, residual=res, z=z)
            assert torch.equal(got.cpu(), ref) and torch.equal(z.cpu(), far.expand(rows, N))
            if C % 16 == 0:
                sw.swin_block_linear_forward_q8(h, *dev(x8, sx, w8, sc, far), got8, residual=res)
                assert torch.equal(got8.cpu(), ref)
        sw.swin_block_linear_sync_status(h)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(1, 64, 264), (40, 64, 264), (300, 1032, 2056), (2500, 512, 1024), (4000, 96, 264)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradient_far_from_zero(rows, C, N, kind):
    """dz is dy or 0, exactly: what is left are the products' roundings."""
    x, w, _, _, dy = make(rows, C, N, seed=24)
    z = torch.tensor(FAR).repeat(N // 8).to(BF).expand(rows, N).contiguous()
    dz = dy * (z > 0)
    ref, tol = backward_ref(x, w, None, dz, "none")
    g = dict(dx=nans(rows, C), dW=nans(N, C), db=nans(N))
    with linear(C, N, kind) as h:
        sw.swin_block_linear_backward(h, *dev(x, w, dy), g["dx"], g["dW"], g["db"], z=dev(z))
        sw.swin_block_linear_sync_status(h)
    for k in ref:
        close(g[k], ref[k], tol[k])
    assert not g["dW"][z[0] < 0].any() and not g["db"][z[0] < 0].any()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,behind,C,N", [(1, 4, 192, 520), (77, 51, 192, 520), (300, 100, 192, 520),
                                             (385, 127, 2960, 400), (2500, 60, 512, 1024)])
def test_in_place_and_rows_behind_the_batch(rows, behind, C, N):
    x, w, b, r, dy = make(rows + behind, C, N, seed=4)
    _, out, _, eo = forward_ref(x[:rows], w, b, r[:rows], "gelu")
    xd, wd, bd, rd, yd = dev(x, w, b, r, dy)
    z, dx = torch.full_like(rd, 7.0), torch.full_like(xd, 7.0)
    (x8, sx), (w8, sc) = quantise(xd), quantise(wd)
    r8 = rd.clone()
    with linear(C, N, "gelu") as h:
        sw.swin_block_linear_forward(h, xd[:rows], wd, bd, rd[:rows], residual=rd[:rows], z=z[:rows])
        again = dev(r)
        sw.swin_block_linear_forward(h, xd[:rows], wd, bd, again[:rows], residual=again[:rows])
        sw.swin_block_linear_forward_q8(h, x8[:rows], sx[:rows], w8, sc, bd, r8[:rows], residual=r8[:rows])
        sw.swin_block_linear_backward(h, xd[:rows], wd, yd[:rows], dx[:rows], nans(N, C), nans(N), z=z[:rows])
        sw.swin_block_linear_sync_status(h)
    close(rd[:rows], out, eo)
    assert torch.equal(rd, again)
    assert torch.equal(rd[rows:].cpu(), r[rows:]) and torch.equal(r8[rows:].cpu(), r[rows:])
    assert (z[rows:] == 7).all() and (dx[rows:] == 7).all() and not (z[:rows] == 7).all()


@pytest.mark.gpu
def test_empty_batch():
    C, N = 96, 256
    x, w, b, _, _ = make(0, C, N)
    xd, wd, bd = dev(x, w, b)
    wide = torch.empty(0, N, dtype=BF, device=DEV)
    dW, db = nans(N, C), nans(N)
    with linear(C, N, "gelu") as h:
        sw.swin_block_linear_forward(h, xd, wd, bd, wide.clone(), z=wide.clone())
        sw.swin_block_linear_backward(h, xd, wd, wide, xd.clone(), dW, db, z=wide.clone())
        sw.swin_block_linear_sync_status(h)
    assert not dW.any() and not db.any()


@pytest.mark.gpu
def test_leading_axes():
    """x [..., C] of any number of axes."""
    x, w, b, _, dy = make(2 * 3 * 5, 64, 96, seed=5)
    xd, wd, bd, yd = dev(x, w, b, dy)
    shaped = xd.view(2, 3, 5, 64)
    out, z, dx = nans(2, 3, 5, 96), nans(2, 3, 5, 96), nans(2, 3, 5, 64)
    with linear(64, 96, "gelu") as h:
        sw.swin_block_linear_forward(h, shaped, wd, bd, out, z=z)
        sw.swin_block_linear_backward(h, shaped, wd, yd.view(2, 3, 5, 96), dx, nans(96, 64), z=z)
        sw.swin_block_linear_sync_status(h)
    _, ref, _, eo = forward_ref(x, w, b, None, "gelu")
    close(out.view(-1, 96), ref, eo)
    ref, tol = backward_ref(x, w, z.view(-1, 96).cpu(), dy, "gelu")
    close(dx.view(-1, 64), ref["dx"], tol["dx"], 2 * HALF)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(1, 256, 640), (40, 256, 640), (700, 4096, 120), (1000, 8192, 1032),
                                      (2500, 512, 2048), (3000, 1024, 1000)])
def test_streams_and_captured_graphs_share_nothing(rows, C, N):
    x, w, b, _, dy = make(rows, C, N, seed=5)
    x2, _, _, _, dy2 = make(rows, C, N, seed=6)
    wd, bd = dev(w, b)
    a, c = dev(x, dy), dev(x2, dy2)
    with linear(C, N, "gelu") as h:
        def call(x, dy):
            o = [nans(rows, N), nans(rows, N), nans(rows, C), nans(N, C), nans(N)]
            sw.swin_block_linear_forward(h, x, wd, bd, o[0], z=o[1])
            sw.swin_block_linear_backward(h, x, wd, dy, o[2], o[3], o[4], z=o[1])
            return o

        same = lambda o, w: all(torch.equal(i, j) for i, j in zip(o, w))  # noqa: E731
        want, want2 = call(*a), call(*c)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for k in range(6):
            with torch.cuda.stream(streams[k % 2]):
                got.append(call(*(a if k % 2 else c)))
        torch.cuda.synchronize()
        assert all(same(o, want if k % 2 else want2) for k, o in enumerate(got))
        graphs = []
        for t in (a, c):
            bufs = [v.clone() for v in t]
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                o = call(*bufs)
            graphs.append((gr, bufs, o))
        for v, t in zip(graphs[0][1], c):
            v.copy_(t)
        torch.cuda.synchronize()
        for (gr, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        eager = call(*a)
        torch.cuda.synchronize()
        sw.swin_block_linear_sync_status(h)
        assert same(graphs[0][2], want2) and same(graphs[1][2], want2) and same(eager, want)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(3, 72, 136), (60, 152, 1736), (128, 2048, 264), (300, 1032, 256), (4067, 136, 1000)])
@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_backwards_back_to_back(rows, C, N, kind):
    """Calls on one stream with nothing in between, in eager order and in a graph: a
    call's kernels may run beside each other, but not into the next call's, which writes
    the same workspace (dz, partial sums)."""
    sets = []
    for seed in (30, 31, 32):
        x, w, b, _, dy = make(rows, C, N, seed=seed)
        sets.append(dev(x, w, dy) + [None if kind == "none" else dev(stored_z(x, w, b))])
    out = lambda: [nans(rows, C), nans(N, C), nans(N)]  # noqa: E731
    with linear(C, N, kind) as h:
        def call(s, o):
            sw.swin_block_linear_backward(h, s[0], s[1], s[2], *o, z=s[3])

        want = [out() for _ in sets]
        for s, o in zip(sets, want):
            call(s, o)
            torch.cuda.synchronize()
        got, graphed = ([out() for _ in range(24)] for _ in "eg")
        torch.cuda.synchronize()
        for i, o in enumerate(got):
            call(sets[i % 3], o)
        gr = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(gr):
            for i, o in enumerate(graphed):
                call(sets[i % 3], o)
        gr.replay()
        sw.swin_block_linear_sync_status(h)
        torch.cuda.synchronize()
        for i in range(24):
            for a, b, c in zip(got[i], graphed[i], want[i % 3]):
                assert torch.equal(a, c) and torch.equal(b, c), i
        del gr
        torch.cuda.synchronize()


@pytest.mark.gpu
def test_first_call_of_a_handle_captured():
    """A handle's first call may be the captured one (here with a workspace)."""
    rows, C, N = 1000, 8192, 1032
    x, w, b, r, _ = make(rows, C, N, seed=11)
    _, ref, _, eo = forward_ref(x, w, b, r, "silu")
    xd, wd, bd, rd = dev(x, w, b, r)
    out = torch.zeros(rows, N, dtype=BF, device=DEV)
    with linear(C, N, "silu") as h:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            sw.swin_block_linear_forward(h, xd, wd, bd, out, residual=rd)
        for _ in range(2):
            gr.replay()
        sw.swin_block_linear_sync_status(h)
        assert sw.swin_block_linear_last_launches(h) == 2   # (the second adds the partial tiles)
        close(out, ref, eo)
        del gr
        torch.cuda.synchronize()


FIRST = """
import torch
from vision_transformer_shifted_gb300 import binding as sw
rows, C, N = %d, %d, %d
n = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, w, b, y, g, bt = n(rows, C), n(N, C), n(N), n(rows, N), n(C), n(C)
norm, z, out, dx, ds, dW, db = n(rows, C), n(rows, N), n(rows, N), n(rows, C), n(rows, C), n(N, C), n(N)
dg = torch.empty(2, C, device="cuda")
h, ln = sw.swin_block_linear_create(C, N, sw.BLOCK_LINEAR_GELU), sw.swin_block_layernorm_create(C, 1e-5)
def call():
    sw.swin_block_layernorm_forward(ln, x, g, bt, norm)
    sw.swin_block_linear_forward(h, norm, w, b, out, z=z)
    sw.swin_block_linear_backward(h, norm, w, y, dx, dW, db, z=z)
    sw.swin_block_layernorm_backward(ln, x, g, dx, ds, dg[0], dg[1])
    return [t.clone() for t in (norm, z, out, dx, dW, db, ds, dg)]
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    got = call()
gr.replay()
torch.cuda.synchronize()
sw.swin_block_linear_sync_status(h)
assert all(torch.equal(a, b) for a, b in zip(got, call()))
del gr
torch.cuda.synchronize()
sw.swin_block_linear_destroy(h)
sw.swin_block_layernorm_destroy(ln)
print("same")
"""


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(1, 256, 640), (40, 4096, 640), (300, 1032, 2056), (2500, 512, 1024)])
def test_first_call_of_a_process_captured(rows, C, N):
    """The first call a process makes at all may be a captured one: what the library
    asks the device, or loads, on the way is allowed there."""
    done = subprocess.run([sys.executable, "-c", FIRST % (rows, C, N)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip() == "same", done.stderr[-2000:]


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """z, out and dz of more than 2^31 elements: the last rows, and those around the
    2^31st element, forward and backward."""
    rows, C, N = 33000, 136, 65536
    g = torch.Generator(device=DEV).manual_seed(5)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)  # noqa: E731
    x, w, b, dy = n(rows, C), n(N, C, std=C ** -0.5), n(N, std=0.3), n(rows, N)
    out, z = nans(rows, N), nans(rows, N)
    some = [0, 32766, 32767, 32768, 32769, rows - 1]
    with linear(C, N, "gelu") as h:
        sw.swin_block_linear_forward(h, x, w, b, out, residual=dy, z=z)
        ref, o, ez, eo = forward_ref(x[some].cpu(), w.cpu(), b.cpu(), dy[some].cpu(), "gelu")
        close(z[some], ref, ez)
        close(out[some], o, eo)
        del out
        dx, dW, db = nans(rows, C), nans(N, C), nans(N)
        sw.swin_block_linear_backward(h, x, w, dy, dx, dW, db, z=z)
        sw.swin_block_linear_sync_status(h)
    ref, tol = backward_ref(x[some].cpu(), w.cpu(), z[some].cpu(), dy[some].cpu(), "gelu")
    close(dx[some], ref["dx"], tol["dx"], 2 * HALF)
    few = [0, 1, 30001, N - 1]   # columns of all rows
    ref, tol = backward_ref(x.cpu(), w[few].cpu(), z[:, few].cpu(), dy[:, few].cpu(), "gelu")
    close(dW[few], ref["dW"], tol["dW"], 2 * HALF)
    close(db[few], ref["db"], tol["db"])


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 5, 200])
def test_weights_past_32_bits(rows):
    """W and dW of more than 2^31 elements: outputs on both sides of that, dx over all of
    W's rows, dW around the 2^31st element and at its end."""
    C, N = 65536, 32776
    g = torch.Generator(device=DEV).manual_seed(rows)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)  # noqa: E731
    x, w, b, dy = n(rows, C), n(N, C, std=C ** -0.5), n(N, std=0.3), n(rows, N)
    some = [0, 1, 32766, 32767, 32768, 32769, N - 1]
    out, dx, dW, db = nans(rows, N), nans(rows, C), nans(N, C), nans(N)
    with linear(C, N) as h:
        sw.swin_block_linear_forward(h, x, w, b, out)
        sw.swin_block_linear_backward(h, x, w, dy, dx, dW, db)
        sw.swin_block_linear_sync_status(h)
    _, ref, _, tol = forward_ref(x, w[some], b[some], None, "none")
    close(out[:, some], ref.cpu(), tol.cpu())
    ref, tol = backward_ref(x, w[some], None, dy[:, some], "none")
    close(dW[some], ref["dW"].cpu(), tol["dW"].cpu())
    close(db[some], ref["db"].cpu(), tol["db"].cpu())
    at = [0, 1, 255, 256, 40000, C - 1]   # columns of dx, over all of W's rows
    ref, tol = backward_ref(x[:, at], w[:, at], None, dy, "none")
    close(dx[:, at], ref["dx"].cpu(), tol["dx"].cpu())


@pytest.mark.gpu
def test_simulated_allocation_failure_then_a_normal_call():
    rows, C, N = 1000, 8192, 1032
    x, w, b, _, dy = make(rows, C, N, seed=12)
    xd, wd, bd, yd = dev(x, w, b, dy)
    out, dx, dW = torch.full_like(yd, 5.0), torch.full_like(xd, 5.0), nans(N, C)
    with linear(C, N, "gelu") as h:
        with env("SWIN_WATTN_FAIL_ALLOC"):
            for call in (lambda: sw.swin_block_linear_forward(h, xd, wd, bd, out),
                         lambda: sw.swin_block_linear_backward(h, xd, wd, yd, dx, dW, z=yd)):
                with pytest.raises(sw.SwinWAttnError) as ei:
                    call()
                assert ei.value.code == sw.ENOMEM
        torch.cuda.synchronize()
        assert (out == 5).all() and (dx == 5).all()
        sw.swin_block_linear_forward(h, xd, wd, bd, out)
        sw.swin_block_linear_sync_status(h)
    _, ref, _, eo = forward_ref(x, w, b, None, "gelu")
    close(out, ref, eo)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C,N", [(1, 96, 256), (70, 264, 520), (300, 1032, 2056), (700, 4096, 120), (1000, 8192, 1032),
                                      (2500, 512, 2048)])
def test_guard_bands_stay_intact_and_catch_an_overwrite(rows, C, N):
    x, w, b, r, dy = make(rows, C, N, seed=13)
    xd, wd, bd, rd, yd = dev(x, w, b, r, dy)
    with env("SWIN_WATTN_DEBUG"), linear(C, N, "silu") as h:   # the bands are read back after each call
        sw.swin_block_linear_forward(h, xd, wd, bd, nans(rows, N), residual=rd)
        back = lambda: sw.swin_block_linear_backward(h, xd, wd, yd, nans(rows, C), nans(N, C), nans(N), z=rd)  # noqa: E731
        back()
        for side in (0, 1):
            sw.swin_block_linear_test_corrupt_workspace(h, side)
            with pytest.raises(sw.SwinWAttnError) as ei:
                back()
            assert ei.value.code == sw.ECORRUPT


@pytest.mark.gpu
def test_two_host_threads_compute_what_one_does():
    """A handle a thread at once: every result is the one that the call gives alone."""
    import threading
    wrong, data = [], []
    for rows, C, N in ((1, 1000, 640), (128, 256, 1024), (700, 4096, 120), (3001, 96, 384), (1300, 2048, 2056)):
        x, w, b, _, dy = dev(*make(rows, C, N, seed=14))
        z = (x @ w.t())

        def call(h, x=x, w=w, b=b, dy=dy, z=z):
            o = [torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)]
            sw.swin_block_linear_forward(h, x, w, b, o[0], residual=dy)
            sw.swin_block_linear_backward(h, x, w, dy, *o[1:], z=z)
            return o

        with linear(C, N, "gelu") as h:
            data.append((C, N, call, call(h)))
    torch.cuda.synchronize()

    def work(C, N, call, want):
        try:
            stream = torch.cuda.Stream()
            with linear(C, N, "gelu") as h, torch.cuda.stream(stream):
                for _ in range(50):
                    got = call(h)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        wrong.append((C, N))
        except Exception as e:
            wrong.append((C, N, e))

    threads = [threading.Thread(target=work, args=a) for a in data]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


# ---- as a block uses it ----------------------------------------------------------------

def layer_norm(s, gamma, beta, eps=1e-5):
    mu = s.mean(-1, keepdim=True)
    return (s - mu) / ((s - mu).pow(2).mean(-1, keepdim=True) + eps).sqrt() * gamma + beta


@pytest.mark.gpu
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("rows,C,ratio", [(3136, 96, 4), (333, 256, 4), (1, 512, 4)])
def test_second_sub_layer_of_a_block_and_its_gradients(rows, C, ratio, post):
    """The MLP sub-layer out of these operators, forward and backward, against
    autograd in float64.  V1: s = z + branch, y = s + W2 GELU(W1 LN(s)); V2: y = z +
    LN(W2 GELU(W1 z)).  Every stored value on the way (n, h, dh, dz, dn) adds a
    relative 2^-8 at most, averaged over the sums that read it."""
    R = ratio * C
    g = torch.Generator().manual_seed(rows + C + post)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)  # noqa: E731
    z, branch, dy = n(rows, C), n(rows, C), n(rows, C)
    p = dict(gamma=(1 + 0.1 * torch.randn(C, generator=g)).to(BF), beta=n(C, std=0.1), W1=n(R, C, std=C ** -0.5),
             b1=n(R, std=0.1), W2=n(C, R, std=R ** -0.5), b2=n(C, std=0.1))
    zd, brd, yd = dev(z, branch, dy)
    d = {k: v.to(DEV) for k, v in p.items()}
    new = lambda *s: nans(*s)  # noqa: E731
    gr = dict(W1=new(R, C), b1=new(R), W2=new(C, R), b2=new(C), gamma=torch.empty(C, device=DEV),
              beta=torch.empty(C, device=DEV))
    s, norm, pre, hid, out = new(rows, C), new(rows, C), new(rows, R), new(rows, R), new(rows, C)
    dhid, dnorm, ds = new(rows, R), new(rows, C), new(rows, C)
    ln = sw.swin_block_layernorm_create(C, 1e-5)
    with linear(C, R, "gelu") as l1, linear(R, C) as l2:
        if not post:
            sw.swin_block_layernorm_forward(ln, zd, d["gamma"], d["beta"], norm, residual=brd, out_sum=s)
            sw.swin_block_linear_forward(l1, norm, d["W1"], d["b1"], hid, z=pre)
            sw.swin_block_linear_forward(l2, hid, d["W2"], d["b2"], out, residual=s)
            sw.swin_block_linear_backward(l2, hid, d["W2"], yd, dhid, gr["W2"], gr["b2"])
            sw.swin_block_linear_backward(l1, norm, d["W1"], dhid, dnorm, gr["W1"], gr["b1"], z=pre)
            sw.swin_block_layernorm_backward(ln, s, d["gamma"], dnorm, ds, gr["gamma"], gr["beta"], dsum=yd)
            start = (z.float() + branch.float()).to(BF)
        else:
            s = zd
            sw.swin_block_linear_forward(l1, s, d["W1"], d["b1"], hid, z=pre)
            sw.swin_block_linear_forward(l2, hid, d["W2"], d["b2"], norm)
            sw.swin_block_layernorm_forward_post(ln, norm, d["gamma"], d["beta"], s, out)
            dnorm2 = new(rows, C)
            sw.swin_block_layernorm_backward(ln, norm, d["gamma"], yd, dnorm2, gr["gamma"], gr["beta"])
            sw.swin_block_linear_backward(l2, hid, d["W2"], dnorm2, dhid, gr["W2"], gr["b2"])
            sw.swin_block_linear_backward(l1, s, d["W1"], dhid, dnorm, gr["W1"], gr["b1"], z=pre)
            ds = dnorm + yd
            start = z
        sw.swin_block_linear_sync_status(l1)
        sw.swin_block_linear_sync_status(l2)
    sw.swin_block_layernorm_destroy(ln)
    leaves = {k: v.double().requires_grad_() for k, v in p.items()}
    ss = start.double().requires_grad_()

    def mlp(t):
        return torch.nn.functional.gelu(t @ leaves["W1"].t() + leaves["b1"]) @ leaves["W2"].t() + leaves["b2"]

    if post:
        y = ss + layer_norm(mlp(ss), leaves["gamma"], leaves["beta"])
    else:
        y = ss + mlp(layer_norm(ss, leaves["gamma"], leaves["beta"]))
    (y * dy.double()).sum().backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, y.detach()) <= 3 * HALF
    assert rel(ds, ss.grad) <= 5 * HALF
    for k, v in leaves.items():
        assert rel(gr[k], v.grad) <= 6 * HALF, k


@pytest.mark.gpu
@pytest.mark.parametrize("C,H", [(96, 28), (192, 8)])
def test_merging_step_out_of_norm_and_linear(C, H):
    """swin_merge_forward's steps: the 2 x 2 neighbourhoods, LN over 4C, the linear
    layer without bias; here each of them has a gradient."""
    g = torch.Generator().manual_seed(C)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF).to(DEV)  # noqa: E731
    x, gamma, beta, W = n(2, H, H, C), n(4 * C, std=0.1) + 1, n(4 * C, std=0.1), n(2 * C, 4 * C, std=(4 * C) ** -0.5)
    want, out = nans(2, H // 2, H // 2, 2 * C), nans(2, H // 2, H // 2, 2 * C)
    m = sw.swin_merge_create(C)
    sw.swin_merge_forward(m, x, gamma, beta, W, want)
    sw.swin_merge_destroy(m)
    cat = torch.cat([x[:, i::2, j::2] for j in (0, 1) for i in (0, 1)], -1).contiguous()
    norm = torch.empty_like(cat)
    ln = sw.swin_block_layernorm_create(4 * C, 1e-5)
    with linear(4 * C, 2 * C) as h:
        sw.swin_block_layernorm_forward(ln, cat, gamma, beta, norm)
        sw.swin_block_linear_forward(h, norm, W, None, out)
        sw.swin_block_linear_sync_status(h)
    sw.swin_block_layernorm_destroy(ln)
    # (both round the norm and the result: two roundings apart each)
    assert float((out.double() - want.double()).norm() / want.double().norm()) <= 2 * HALF


@pytest.mark.gpu
def test_served_in_eight_bits():
    """Norm to e4m3, then the 8-bit layer: from the codes and scales themselves."""
    rows, C, N = 333, 256, 640
    x, w, b, r, _ = make(rows, C, N, seed=7)
    gamma, beta = (1 + 0.1 * torch.randn(C, generator=torch.Generator().manual_seed(1))).to(BF), torch.zeros(C).to(BF)
    codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.empty(rows, device=DEV)
    w8, sc = quantise(w)
    out = nans(rows, N)
    ln = sw.swin_block_layernorm_create(C, 1e-5)
    with linear(C, N, "silu") as h:
        sw.swin_block_layernorm_forward_q8(ln, dev(x), dev(gamma), dev(beta), codes, scales)
        sw.swin_block_linear_forward_q8(h, codes, scales, *dev(w8, sc, b), out, residual=dev(r))
        sw.swin_block_linear_sync_status(h)
    sw.swin_block_layernorm_destroy(ln)
    _, ref, _, eo = forward_ref(codes.cpu().double() * scales.cpu().double()[:, None],
                                w8.double() * sc.double()[:, None], b, r, "silu")
    close(out, ref, eo)
