"""Layer norm of the residual stream (include/swin_layernorm.h).

CPU (not gpu): the arguments each entry point refuses, and the gradient
formula against central differences.  GPU: forward (bf16, post-norm and e4m3)
and backward against the formula in float64, at widths on each side of the row
layouts (part of a warp, a block), odd row counts, in place, rows of zeros, of
one value, far from zero, of infinities and NaN, on another stream, captured
and replayed.

Tolerances: a rounding to bf16 is off by at most 2^-8 of the value (half a
step), to e4m3 by 2^-4 or, below its smallest normal number, half of 2^-9.
The fp32 sums have at most 16384 terms in chains of at most some 100, so that a
row's statistics are good to FP = 2^-15, n to FP (|n| + 1/16) (its mean is a
sum of terms of order one) and, since s - mu is one fp32 subtraction whose
operands may be larger than itself, to 2^-22 (|s| + |mu|) r beside.  (The sums are
of s - p, p the mean of the row's first eight values: k standard deviations from
the row's mean, k below 2 in random rows.  Rows with their spread in those eight
values have bounds of their own, with k in them.)
"""
import ctypes

import pytest
import torch

from vision_transformer_shifted_gb300 import binding as sw

DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF, FP, SUB = 2.0 ** -8, 2.0 ** -15, 2.0 ** -22
EPS = 1e-5


def normalise(s, eps=EPS):
    """n, r and the bound on n's error, float64."""
    s = s.double()
    mu = s.mean(-1, keepdim=True)
    r = 1 / ((s - mu).pow(2).mean(-1, keepdim=True) + eps).sqrt()
    n = (s - mu) * r
    return n, r, FP * (n.abs() + 1 / 16) + SUB * (s.abs() + mu.abs()) * r


def reference(x, residual, gamma, beta, eps=EPS):
    """s (bf16), y and the bound on y's error before it is rounded (float64)."""
    s = x if residual is None else (x.float() + residual.float()).to(BF)
    n, _, e = normalise(s, eps)
    b = torch.zeros(()) if beta is None else beta
    return s, n * gamma.double() + b.double(), e * gamma.double().abs() + FP * b.double().abs()


def gradients(s, gamma, dy, dsum, eps=EPS):
    """dx, dgamma, dbeta in float64 and the bounds on their errors (dx: before it
    is rounded)."""
    n, r, en = normalise(s, eps)
    gamma, dy = gamma.double(), dy.double()
    a = dy * gamma
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    dx = r * (a - mean(a) - n * mean(a * n))
    err = r * (FP * (a.abs() + mean(a.abs()) + n.abs() * mean((a * n).abs())) + en * mean((a * n).abs())
               + n.abs() * mean(a.abs() * en))
    if dsum is not None:
        dx, err = dx + dsum.double(), err + FP * dsum.double().abs()
    return (dx, (dy * n).sum(0), dy.sum(0)), (err, (dy.abs() * (en + FP * n.abs())).sum(0), FP * dy.abs().sum(0))


def inputs(rows, C, residual=True, seed=0):
    """x (with a mean of its own a row), residual, gamma, beta, dy."""
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 4099 + C)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((n(rows, C) * 2 + 3 * n(rows, 1)).to(BF), n(rows, C).to(BF) if residual else None,
            (1 + 0.2 * n(C)).to(BF), (0.3 * n(C)).to(BF), n(rows, C).to(BF))


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


class layernorm:
    def __init__(self, C, eps=EPS):
        self.args = C, eps

    def __enter__(self):
        self.h = sw.swin_block_layernorm_create(*self.args)
        return self.h

    def __exit__(self, *exc):
        sw.swin_block_layernorm_destroy(self.h)


def close(got, ref, tol):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got.double()).all()
    assert (err <= tol).all(), float((err - tol).max())


def close_codes(codes, scales, y, e):
    """Codes and scales of y, whose own error is e."""
    ref = y.abs().amax(-1, keepdim=True) / 448
    worst = e.amax(-1, keepdim=True)
    close(scales[..., None], ref, FP * ref + worst / 448)
    got = codes.float().double().cpu() * scales.double().cpu()[..., None]
    close(got, y, (2.0 ** -4 + FP) * y.abs() + 2.0 ** -10 * ref + 1.1 * (e + worst))


# ---- CPU ---------------------------------------------------------------------------

@pytest.mark.parametrize("C,eps", [(0, 1e-6), (-8, 1e-6), (12, 1e-6), (16392, 1e-6), (64, -1e-6),
                                   (64, float("nan")), (64, float("inf"))])
def test_create_refuses(C, eps):
    h = ctypes.c_void_p(1)
    assert sw.load().swin_block_layernorm_create(ctypes.byref(h), C, eps) == sw.EINVAL
    assert h.value is None
    assert sw.load().swin_block_layernorm_create(None, 64, 1e-6) == sw.EINVAL


P = 1 << 20   # addresses that no refused call reads


def test_forward_refuses():
    lib = sw.load()
    n = 4 * 64 * 2   # bytes of a [4, 64] bf16 tensor
    ok = dict(x=P, residual=P + 4 * n, rows=4, gamma=P + 8 * n, beta=P + 9 * n, out_sum=P + 12 * n, out=P + 16 * n)

    def call(**kw):
        a = {**ok, **kw}
        with layernorm(64) as h:
            h = a.get("h", h)
            args = [h, a["x"], a["residual"], a["rows"], a["gamma"], a["beta"]]
            rc = lib.swin_block_layernorm_forward(*args, a["out_sum"], a["out"], None)
            assert rc == lib.swin_block_layernorm_forward_q8(*args, a["out_sum"], a["out"], P + 32 * n, None)
            if "out_sum" not in kw and kw.get("out") != ok["out_sum"]:
                assert rc == lib.swin_block_layernorm_forward_post(*args, a["out"], None)
        return rc

    assert call(rows=0) == sw.OK
    for bad in (dict(h=None), dict(x=None), dict(gamma=None), dict(out=None), dict(rows=-1), dict(x=P + 8),
                dict(residual=P + 4 * n + 2), dict(gamma=P + 8), dict(beta=P + 2), dict(out=P + 16 * n + 4),
                dict(out_sum=P + 8), dict(residual=None), dict(out=P + 16), dict(out=ok["residual"] + 16),
                dict(out=ok["out_sum"]), dict(out_sum=P + 16), dict(out=ok["gamma"]), dict(out_sum=ok["gamma"]),
                dict(out=ok["beta"]), dict(out_sum=ok["beta"])):
        assert call(**bad) == sw.EINVAL, bad
    with layernorm(64) as h:
        f = lib.swin_block_layernorm_forward_q8
        args = [h, P, None, 4, ok["gamma"], ok["beta"], None]
        for out8, scales in ((ok["out"], None), (ok["out"], P + 4), (P, ok["out"]), (ok["out"], P),
                             (ok["out"], ok["out"]), (ok["out"], ok["gamma"]), (ok["out"], ok["beta"])):
            assert f(*args, out8, scales, None) == sw.EINVAL, (out8, scales)


def test_backward_refuses():
    lib = sw.load()
    n = 4 * 64 * 2
    names = ["s", "gamma", "dy", "dsum", "dx", "dgamma", "dbeta"]
    ok = dict({k: P + 4 * i * n for i, k in enumerate(names)}, rows=4)
    with layernorm(64) as h:
        bads = [dict(h=None), dict(rows=-1)] + [{k: None} for k in names if k not in ("dsum", "dbeta")]
        bads += [{k: ok[k] + 4} for k in names]
        bads += [dict(dx=P), dict(dx=P + 16), dict(dx=ok["dy"] + 16), dict(dx=ok["dsum"] + 16), dict(dx=ok["gamma"])]
        bads += [{o: ok[i]} for o in ("dgamma", "dbeta") for i in names if i != o]
        for bad in bads:
            a = {**ok, **bad}
            assert lib.swin_block_layernorm_backward(a.get("h", h), a["s"], a["rows"], a["gamma"], a["dy"], a["dsum"],
                                                     a["dx"], a["dgamma"], a["dbeta"], None) == sw.EINVAL, bad
    assert lib.swin_block_layernorm_destroy(None) == sw.OK
    assert lib.swin_block_layernorm_last_launches(None) == 0


def test_binding_refuses_other_types_shapes_and_devices():
    x, r, g, b, _ = inputs(4, 64)
    with layernorm(64) as h:
        for kw in (dict(x=x.float()), dict(gamma=g[:32]), dict(beta=b.float()), dict(residual=r[:2]),
                   dict(x=x.t().contiguous().t()), dict(x=x[:, :56].contiguous()), dict()):   # (the last: on the CPU)
            a = {**dict(x=x, gamma=g, beta=b, residual=r), **kw}
            out = torch.empty(4, 64, dtype=BF)
            with pytest.raises(ValueError):
                sw.swin_block_layernorm_forward(h, a["x"], a["gamma"], a["beta"], out, residual=a["residual"])
            with pytest.raises(ValueError):
                sw.swin_block_layernorm_forward_post(h, a["x"], a["gamma"], a["beta"], a["residual"], out)


def test_binding_refuses_more_rows_than_an_int_holds(monkeypatch):
    """2^32 + 1 rows would reach the C side as one."""
    class Tall:   # (what the check asks of a tensor: no such tensor fits here)
        shape, dtype = torch.Size([(1 << 32) + 1, 8]), BF

        def numel(self):
            return 8 * ((1 << 32) + 1)

        def is_contiguous(self):
            return True

        def get_device(self):
            return 0

        def data_ptr(self):
            return 1 << 24

    monkeypatch.setattr(sw, "_current_device", lambda: 0)
    with layernorm(8) as h, pytest.raises(ValueError, match="rows"):
        sw.swin_block_layernorm_forward(h, Tall(), None, None, None)


def test_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    s, gamma, beta, dy, dsum = (torch.randn(*k, generator=g, dtype=torch.float64)
                                for k in ((3, 8), (8,), (8,), (3, 8), (3, 8)))

    def loss(s, gamma, beta):
        return float(((normalise(s)[0] * gamma + beta) * dy).sum() + (s * dsum).sum())

    at = [s, gamma, beta]
    for k, d in enumerate(gradients(s, gamma, dy, dsum)[0]):
        for i in range(at[k].numel()):
            e = torch.zeros(at[k].numel(), dtype=torch.float64)
            e[i] = 1e-5
            up, down = ([t + (z if j == k else 0) for j, t in enumerate(at)]
                        for z in (e.view(at[k].shape), -e.view(at[k].shape)))
            assert abs((loss(*up) - loss(*down)) / 2e-5 - float(d.reshape(-1)[i])) < 1e-6


# ---- GPU ---------------------------------------------------------------------------

SHAPES = [(1, 8), (1, 2048), (3, 16), (33, 40), (257, 96), (70, 192), (19, 520), (9, 1016), (5, 1024), (7, 1032),
          (4, 2744), (3, 4096), (2, 8200), (2, 16384), (10007, 96), (700, 2744)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(rows, C, residual):
    x, r, g, b, _ = inputs(rows, C, residual)
    s, y, e = reference(x, r, g, b)
    xd, rd, gd, bd = dev(x, r, g, b)
    out = torch.full_like(xd, float("nan"))
    out_sum = torch.full_like(xd, float("nan")) if residual else None
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, out, residual=rd, out_sum=out_sum)
        assert sw.swin_block_layernorm_last_launches(h) == 1
        plain = torch.empty_like(out)
        sw.swin_block_layernorm_forward(h, xd, gd, None, plain, residual=rd)
    close(out, y, HALF * y.abs() + 1.01 * e)
    _, y, e = reference(x, r, g, None)
    close(plain, y, HALF * y.abs() + 1.01 * e)
    if residual:
        assert torch.equal(out_sum.cpu(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
def test_forward_post(rows, C):
    x, r, g, b, _ = inputs(rows, C, True, seed=10)
    _, y, e = reference(x, None, g, b)
    y, e = y + r.double(), e + FP * r.double().abs()
    xd, rd, gd, bd = dev(x, r, g, b)
    out = torch.full_like(xd, float("nan"))
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward_post(h, xd, gd, bd, rd, out)
        close(out, y, HALF * y.abs() + 1.01 * e)
        keep = xd.clone()
        sw.swin_block_layernorm_forward_post(h, keep, gd, bd, rd, keep)   # over the branch
        sw.swin_block_layernorm_forward_post(h, xd, gd, bd, rd, rd)       # over the residual
    assert torch.equal(keep, out) and torch.equal(rd, out)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
def test_forward_q8(rows, C):
    residual = C % 16 == 0
    x, r, g, b, _ = inputs(rows, C, residual, seed=1)
    s, y, e = reference(x, r, g, b)
    xd, rd, gd, bd = dev(x, r, g, b)
    codes = torch.full((rows, C), 5.0, device=DEV).to(E4M3)
    scales = torch.full((rows,), float("nan"), device=DEV)
    out_sum = torch.empty_like(xd) if residual else None
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward_q8(h, xd, gd, bd, codes, scales, residual=rd, out_sum=out_sum)
    close_codes(codes, scales, y, e)
    if residual:
        assert torch.equal(out_sum.cpu(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("with_dsum", [True, False])
def test_backward(rows, C, with_dsum):
    s, dsum, g, _, dy = inputs(rows, C, with_dsum, seed=2)
    ref, err = gradients(s, g, dy, dsum)
    sd, md, gd, yd = dev(s, dsum, g, dy)
    new = lambda: (torch.full_like(sd, float("nan")), *(torch.full((C,), float("nan"), device=DEV) for _ in "gb"))  # noqa: E731
    got, again, alone = new(), new(), new()
    with layernorm(C) as h:
        sw.swin_block_layernorm_backward(h, sd, gd, yd, *got, dsum=md)
        assert sw.swin_block_layernorm_last_launches(h) in (1, 2)
        sw.swin_block_layernorm_backward(h, sd, gd, yd, *again, dsum=md)
        sw.swin_block_layernorm_backward(h, sd, gd, yd, *alone[:2], dsum=md)   # without dbeta
    close(got[0], ref[0], HALF * ref[0].abs() + 1.01 * err[0])
    close(got[1], ref[1], err[1])
    close(got[2], ref[2], err[2])
    for a, b in zip(got, again):
        assert torch.equal(a, b)   # a fixed order of summation
    assert torch.equal(got[0], alone[0]) and torch.equal(got[1], alone[1])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [40, 96, 520, 768, 2744])
@pytest.mark.parametrize("mean", [1.0, -300.0, 1000.0, 3e4, 2.0 ** 100])
def test_rows_of_one_value_and_far_from_zero(C, mean):
    """A row of one value has n = 0 whatever its size (y = beta: all its differences
    from its first values are zero); a row of large values with a small spread keeps
    its digits."""
    x, _, g, b, dy = inputs(5, C, False, seed=11)
    x[:3] = mean
    if abs(mean) < 1e6:
        x[3:] = (mean + torch.randn(2, C, generator=torch.Generator().manual_seed(C)) * abs(mean) / 50).to(BF)
    s, y, e = reference(x, None, g, b)
    xd, gd, bd, yd = dev(x, g, b, dy)
    out = torch.empty_like(xd)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, out)
        close(out, y, HALF * y.abs() + 1.01 * e)
        if abs(mean) < 1e6:
            assert ((out[:3].cpu().double() - b.double()).abs() <= HALF * b.double().abs() + 2.0 ** -20).all()
            ref, err = gradients(s, g, dy, None)
            dx, dg, db = torch.empty_like(xd), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
            sw.swin_block_layernorm_backward(h, xd, gd, yd, dx, dg, db)
            close(dx, ref[0], HALF * ref[0].abs() + 1.01 * err[0])
            close(dg, ref[1], err[1])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [8, 96, 520, 2744, 16384])
@pytest.mark.parametrize("where", [slice(3, 4), slice(0, 8)])
def test_a_rows_spread_in_its_first_values(C, where):
    """Large values among the row's first eight, whose mean the sums are taken about:
    it lies k standard deviations from the row's mean, k^2 up to C / 8.

    With u = 2^-24 and at most 40 additions one after the other: the sum of s - p is
    off by 40 u sum|s - p| at most, so mu by 40 u q sigma with q^2 = 1 + k^2; the mean
    square by 41 u q^2 sigma^2, mu's square by 2 k sigma 40 u q sigma <= 80 u q^2
    sigma^2, so var by 122 u q^2 of itself and r by er = 61 u q^2 + 2 u.  n = (s - p) r
    + shift: er |n| + 48 u q.  mean a: 48 u mean|a|; mean(a n), from the sum of a (s - p)
    and mean a: er |mean(a n)| + 50 u (mean|a n| + 2 k mean|a|)."""
    u = 2.0 ** -24
    x, _, g, b, dy = inputs(6, C, False, seed=21)
    x[:, where] = torch.tensor([1000., -700., 50., 3e4, -2e5, 12.]).to(BF)[:, None]
    g_, b_, dy_ = g.double(), b.double(), dy.double()
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    n, r, _ = normalise(x)
    s = x.double()
    k = (mean(s) - mean(s[:, :8])).abs() * r
    q = (1 + k * k).sqrt()
    er = 61 * u * q * q + 2 * u
    en = er * n.abs() + 48 * u * q
    y, ey = n * g_ + b_, en * g_.abs() + 2 * u * (b_.abs() + (n * g_).abs())
    a = dy_ * g_
    ma, mn = mean(a), mean(a * n)
    emn = er * mn.abs() + 50 * u * (mean((a * n).abs()) + 2 * k * mean(a.abs()))
    (dx, dg, db), _ = gradients(x, g, dy, None)
    ex = er * dx.abs() + r * (4 * u * (a.abs() + (n * mn).abs()) + 48 * u * mean(a.abs()) + n.abs() * emn + mn.abs() * en)
    xd, gd, bd, yd = dev(x, g, b, dy)
    out, codes, scales = torch.empty_like(xd), torch.empty(6, C, dtype=E4M3, device=DEV), torch.empty(6, device=DEV)
    got = torch.empty_like(xd), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, out)
        sw.swin_block_layernorm_forward_q8(h, xd, gd, bd, codes, scales)
        sw.swin_block_layernorm_backward(h, xd, gd, yd, *got)
    close(out, y, HALF * y.abs() + 1.01 * ey)
    close_codes(codes, scales, y, ey)
    close(got[0], dx, HALF * dx.abs() + 1.01 * ex)
    close(got[1], dg, (dy_.abs() * (en + 8 * u * n.abs())).sum(0))
    close(got[2], db, 8 * u * dy_.abs().sum(0))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [8, 96, 520, 768, 2744, 4096, 8200, 16384])
@pytest.mark.parametrize("size", [16.0, 300.0, -30000.0])
def test_statistics_do_not_depend_on_where_a_large_channel_lies(C, size):
    """One channel far above the others, wherever it lies: n in fp32, as dgamma gives it
    for one row and dy = 1, and the e4m3 form's scale, max |n| / 448.

    With u = 2^-24 and at most 40 additions one after the other, sums about a pivot k
    standard deviations from the row's mean leave r off by 61 u (1 + k^2) + 2 u, and n by as
    much of itself and 48 u sqrt(1 + k^2) (the test above).  k^2 is at most two, whatever the
    row's first values are: else the sums are taken again about the mean."""
    u = 2.0 ** -24
    one, zero = torch.ones(C).to(BF), torch.zeros(C).to(BF)
    with layernorm(C) as h:
        for at in sorted({0, 5, 8 % C, C // 2, C - 1}):
            x = inputs(1, C, False, seed=at)[0]
            x[0, at] = size
            n = normalise(x)[0]
            en = (61 * 3 + 2) * 1.01 * u * n.abs() + 48 * 1.01 * 3 ** 0.5 * u
            xd, gd, bd = dev(x, one, zero)
            dg = torch.empty(C, device=DEV)
            sw.swin_block_layernorm_backward(h, xd, gd, gd.view(1, C), torch.empty_like(xd), dg)
            close(dg[None], n, en)   # (1.01: the sums that decide are rounded too)
            for rows in (1, 200):
                codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.empty(rows, device=DEV)
                sw.swin_block_layernorm_forward_q8(h, xd.expand(rows, C).contiguous(), gd, bd, codes, scales)
                i = int(n.abs().argmax())
                close(scales, (n.abs()[0, i] / 448).expand(rows), (en[0, i] / 448 + 2 * u * n.abs()[0, i] / 448).expand(rows))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [8, 40, 96, 520, 768, 2744, 8200, 16384])
@pytest.mark.parametrize("rows", [37, 400])
def test_rows_beside_one_with_a_large_first_channel_keep_their_bits(rows, C):
    """Rows share warps, groups and blocks with others; each has statistics of its own,
    also where a neighbour's are taken twice, and in place."""
    x, r, g, b, dy = inputs(rows, C, True, seed=25)
    big = x.clone()
    big[5, 0] = big[rows - 1, 3] = 30000.0
    big[7, 2] = float("nan")
    rest = [i for i in range(rows) if i not in (5, 7, rows - 1)]
    rd, gd, bd, yd = dev(r, g, b, dy)

    def call(x, h):
        x, o = x.to(DEV), [torch.empty(rows, C, dtype=BF, device=DEV) for _ in range(4)]
        codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.empty(rows, device=DEV)
        sw.swin_block_layernorm_forward(h, x, gd, bd, o[0], residual=rd, out_sum=o[1])
        sw.swin_block_layernorm_forward_post(h, x, gd, bd, rd, o[2])
        sw.swin_block_layernorm_forward_q8(h, x, gd, bd, codes, scales)
        sw.swin_block_layernorm_backward(h, x, gd, yd, o[3], torch.empty(C, device=DEV), dsum=rd)
        over, into = x.clone(), rd.clone()
        sw.swin_block_layernorm_forward(h, over, gd, bd, into, residual=into, out_sum=over)
        assert torch.equal(into.nan_to_num(7.0), o[0].nan_to_num(7.0))
        assert torch.equal(over.nan_to_num(7.0), o[1].nan_to_num(7.0))
        return *o, codes.float(), scales

    with layernorm(C) as h:
        alone, beside = call(x, h), call(big, h)
    for p, q in zip(alone, beside):
        assert torch.equal(p[rest], q[rest])
    for q in beside[:1] + beside[2:]:
        assert q[7].isnan().all() and torch.isfinite(q[5]).all()
    some = [5, rows - 1]
    _, y, e = reference(big[some], r[some], g, b)
    close(beside[0][some], y, HALF * y.abs() + 1.01 * e)
    ref, err = gradients(big[some], g, dy[some], r[some])
    close(beside[3][some], ref[0], HALF * ref[0].abs() + 1.01 * err[0])


@pytest.mark.gpu
def test_rows_past_32_bits_of_elements():
    """rows * C > 2^31: rows at the beginning, around the 2^31st element and at the
    end; the parameters' sums over all of them.  In fp32: some 863 rows a block one
    after the other and 152 partial rows, each addition off by 2^-24 at most."""
    C, rows = 16384, (1 << 17) + 5
    gen = torch.Generator(device=DEV).manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF)  # noqa: E731
    s, dy, g, b = n(rows, C), n(rows, C), 1 + 0.2 * n(C), n(C)
    out = torch.full_like(s, float("nan"))
    dg, db = torch.full((C,), float("nan"), device=DEV), torch.full((C,), float("nan"), device=DEV)
    codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.full((rows,), float("nan"), device=DEV)
    some = [0, 1, 65535, 131070, 131071, 131072, 131073, rows - 1]
    _, y, e = reference(s[some].cpu(), None, g.cpu(), b.cpu())
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward_q8(h, s, g, b, codes, scales)
        close_codes(codes[some], scales[some], y, e)
        sw.swin_block_layernorm_forward(h, s, g, b, out)
        close(out[some], y, HALF * y.abs() + 1.01 * e)
        sw.swin_block_layernorm_forward_post(h, s, g, b, dy, out)
        y, e = y + dy[some].cpu().double(), e + FP * dy[some].cpu().double().abs()
        close(out[some], y, HALF * y.abs() + 1.01 * e)
        sw.swin_block_layernorm_backward(h, s, g, dy, out, dg, db)
    ref, err = gradients(s[some].cpu(), g.cpu(), dy[some].cpu(), None)
    close(out[some], ref[0], HALF * ref[0].abs() + 1.01 * err[0])
    ref, size, tol = torch.zeros(2, C, dtype=torch.float64), torch.zeros(2, C, dtype=torch.float64), torch.zeros(2, C, dtype=torch.float64)
    for i in range(0, rows, 8192):
        sl, dl = s[i:i + 8192], dy[i:i + 8192]
        r_, e_ = gradients(sl, g, dl, None)
        ref += torch.stack(r_[1:]).cpu()
        tol += torch.stack(e_[1:]).cpu()
        nn = normalise(sl)[0]
        size += torch.stack([(dl.double() * nn).abs().sum(0), dl.double().abs().sum(0)]).cpu()
    chain = (863 + 152) * 2.0 ** -24
    close(dg, ref[0], chain * size[0] + tol[0])
    close(db, ref[1], chain * size[1] + tol[1])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 2744])
def test_in_place(C):
    x, r, g, b, dy = inputs(37, C, True, seed=3)
    s, y, e = reference(x, r, g, b)
    xd, rd, gd, bd, yd = dev(x, r, g, b, dy)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, xd, residual=rd, out_sum=rd)
        close(xd, y, HALF * y.abs() + 1.01 * e)
        assert torch.equal(rd.cpu(), s)
        ref, err = gradients(s, g, dy, x)
        gg, gb = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        one, two = yd.clone(), x.to(DEV)
        sw.swin_block_layernorm_backward(h, rd, gd, one, one, gg, gb, dsum=two)
        close(one, ref[0], HALF * ref[0].abs() + 1.01 * err[0])
        sw.swin_block_layernorm_backward(h, rd, gd, yd, two, gg, gb, dsum=two)
        assert torch.equal(one, two)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [520, 2744, 8200, 16384])
@pytest.mark.parametrize("rows", [100, 4000])
def test_in_place_gives_the_very_same(rows, C):
    """Wide rows, of which every thread reads the first piece too: the sum over x or
    over the residual, the output over the other."""
    x, r, g, b, _ = dev(*inputs(rows, C, True, seed=22))
    out, s = torch.empty_like(x), torch.empty_like(x)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, x, g, b, out, residual=r, out_sum=s)
        for swap in (False, True):
            one, two = x.clone(), r.clone()
            sw.swin_block_layernorm_forward(h, one, g, b, one if swap else two, residual=two, out_sum=two if swap else one)
            assert torch.equal(one, out if swap else s) and torch.equal(two, s if swap else out)
        post, over = torch.empty_like(x), x.clone()
        sw.swin_block_layernorm_forward_post(h, x, g, b, r, post)
        sw.swin_block_layernorm_forward_post(h, over, g, b, r, over)
        assert torch.equal(over, post)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 2744])
def test_zero_infinite_and_nan_rows(C):
    x, _, g, b, dy = inputs(6, C, False, seed=4)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, C - 1] = float("nan")
    xd, gd, bd, yd = dev(x, g, b, dy)
    out, codes, scales = torch.empty_like(xd), torch.empty(6, C, dtype=E4M3, device=DEV), torch.empty(6, device=DEV)
    dx, dg = torch.empty_like(xd), torch.empty(C, device=DEV)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, out)
        sw.swin_block_layernorm_forward_q8(h, xd, gd, bd, codes, scales)
        sw.swin_block_layernorm_backward(h, xd, gd, yd, dx, dg)
        zero, one = torch.empty_like(codes), torch.empty_like(scales)
        sw.swin_block_layernorm_forward_q8(h, xd, gd, None, zero, one)
    assert torch.equal(out[1].cpu(), b)
    assert not zero[1].float().any() and 0 < float(one[1]) < 1e-30
    assert out[2:4].isnan().all() and codes[2:4].float().isnan().all() and scales[2:4].isnan().all()
    assert dx[2:4].isnan().all() and dg.isnan().all()
    good = [0, 1, 4, 5]
    _, y, e = reference(x[good], None, g, b)
    close(out[good], y, HALF * y.abs() + 1.01 * e)
    close_codes(codes[good], scales[good], y, e)
    ref, err = gradients(x[good], g, dy[good], None)
    close(dx[good], ref[0], HALF * ref[0].abs() + 1.01 * err[0])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 2744])
def test_huge_rows(C):
    """Squared deviations past the largest fp32 number: n = 0."""
    x, _, g, b, _ = inputs(2, C, False, seed=12)
    x[0] = (x[0].float() * 1e30).to(BF)
    xd, gd, bd = dev(x, g, b)
    out = torch.empty_like(xd)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, out)
    assert torch.equal(out[0].cpu(), b)


@pytest.mark.gpu
def test_empty_batch():
    C = 96
    x = torch.empty(0, C, dtype=BF, device=DEV)
    g, gg, gb = torch.ones(C, dtype=BF, device=DEV), torch.full((C,), 3.0, device=DEV), torch.full((C,), 3.0, device=DEV)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, x, g, g, x.clone())
        sw.swin_block_layernorm_forward_post(h, x, g, g, x.clone(), x.clone())
        sw.swin_block_layernorm_backward(h, x, g, x.clone(), x.clone(), gg, gb)
    assert not gg.any() and not gb.any()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [8, 96, 192, 768, 2744])
@pytest.mark.parametrize("rows", [1, 3, 300, 5003])
def test_backward_without_eps(rows, C):
    """eps = 0 and no row of one value: every gradient is finite, whatever part of a
    block the rows leave empty."""
    s, dsum, g, _, dy = inputs(rows, C, rows % 2 == 1, seed=9)
    ref, err = gradients(s, g, dy, dsum, eps=0.0)
    sd, md, gd, yd = dev(s, dsum, g, dy)
    gx, gg, gb = torch.full_like(sd, float("nan")), *(torch.full((C,), float("nan"), device=DEV) for _ in "gb")
    with layernorm(C, 0.0) as h:
        sw.swin_block_layernorm_backward(h, sd, gd, yd, gx, gg, gb, dsum=md)
    close(gx, ref[0], HALF * ref[0].abs() + 1.01 * err[0])
    close(gg, ref[1], err[1])
    close(gb, ref[2], err[2])


@pytest.mark.gpu
def test_rows_behind_the_batch_stay():
    C, rows = 192, 45
    x, r, g, b, dy = dev(*inputs(64, C, True, seed=6))
    out, out_sum, post, dx = (torch.full_like(x, 7.0) for _ in range(4))
    codes, scales = torch.full((64, C), 7.0, device=DEV).to(E4M3), torch.full((64,), 7.0, device=DEV)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, x[:rows], g, b, out[:rows], residual=r[:rows], out_sum=out_sum[:rows])
        sw.swin_block_layernorm_forward_post(h, x[:rows], g, b, r[:rows], post[:rows])
        sw.swin_block_layernorm_forward_q8(h, x[:rows], g, b, codes[:rows], scales[:rows])
        sw.swin_block_layernorm_backward(h, x[:rows], g, dy[:rows], dx[:rows], torch.empty(C, device=DEV),
                                         torch.empty(C, device=DEV))
    for t in (out, out_sum, post, dx, codes.float(), scales):
        assert (t[rows:] == 7).all() and not (t[:rows] == 7).all()


@pytest.mark.gpu
def test_streams_and_captured_graphs_share_nothing():
    """One handle: eager calls on two streams at once and two captured graphs,
    replayed on new inputs while eager calls run, give the eager results."""
    C, rows = 2048, 3000
    s, _, g, _, dy = dev(*inputs(rows, C, False, seed=7))
    s2, _, _, _, dy2 = dev(*inputs(rows, C, False, seed=8))
    with layernorm(C) as h:
        def call(s, dy):
            o = torch.empty_like(s), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
            sw.swin_block_layernorm_backward(h, s, g, dy, *o)
            return o

        def same(a, b):
            return all(torch.equal(p, q) for p, q in zip(a, b))

        want, want2 = call(s, dy), call(s2, dy2)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for k in range(6):
            with torch.cuda.stream(streams[k % 2]):
                got.append(call(*((s, dy) if k % 2 else (s2, dy2))))
        torch.cuda.synchronize()
        for k, o in enumerate(got):
            assert same(o, want if k % 2 else want2)
        graphs = []
        for a in ((s, dy), (s2, dy2)):
            bufs = [t.clone() for t in a]
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                o = call(*bufs)
            graphs.append((gr, bufs, o))
        for b, t in zip(graphs[0][1], (s2, dy2)):
            b.copy_(t)
        torch.cuda.synchronize()
        for (gr, _, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        eager = call(s, dy)
        torch.cuda.synchronize()
        for _, _, o in graphs:   # both on the second inputs
            assert same(o, want2)
        assert same(eager, want)


@pytest.mark.gpu
def test_two_host_threads_compute_what_one_does():
    """A handle a thread at once: every result is the one that the call gives alone."""
    import threading
    wrong, data = [], []
    for C, rows in ((1000, 8), (16384, 8), (10000, 3), (96, 3001), (2744, 1500)):
        s, _, g, _, dy = dev(*inputs(rows, C, False, seed=C))
        o = torch.empty_like(s), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        with layernorm(C) as h:
            sw.swin_block_layernorm_backward(h, s, g, dy, *o)
        data.append((C, s, g, dy, o))
    torch.cuda.synchronize()

    def work(C, s, g, dy, want):
        try:
            stream = torch.cuda.Stream()
            with layernorm(C) as h, torch.cuda.stream(stream):
                for _ in range(100):
                    o = [torch.empty_like(t) for t in want]
                    sw.swin_block_layernorm_backward(h, s, g, dy, *o)
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(o, want)):
                        wrong.append(C)
        except Exception as e:
            wrong.append((C, e))

    threads = [threading.Thread(target=work, args=a) for a in data]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 256, 2048])
def test_same_as_the_stage_norm(C):
    """The norm between a stage's blocks (eps = 1e-5) is this one: within one
    rounding of each other."""
    x, _, g, b, _ = inputs(100, C, False, seed=13)
    xd, gd, bd = dev(x, g, b)
    one, two = torch.empty_like(xd), torch.empty_like(xd)
    with layernorm(C) as h:
        sw.swin_block_layernorm_forward(h, xd, gd, bd, one)
    sw.swin_stage_norm(xd, gd, bd, two)
    _, y, e = reference(x, None, g, b)
    close(two, y, HALF * y.abs() + 16 * e)
    close(one, two.double().cpu(), 2 * HALF * y.abs() + 17 * e)
