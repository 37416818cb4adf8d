"""RMS norm of the residual stream (include/swin_rms.h).

CPU (not gpu): the arguments each entry point refuses, and the gradient
formula against central differences.  GPU: forward (bf16 and e4m3 output) and
backward against the formula in float64, at widths on each side of the row
layouts (part of a warp, a block), odd row counts, in place, rows of zeros, of
infinities and NaN, on another stream, captured and replayed.

Tolerances: a rounding to bf16 is off by at most 2^-8 of the value (half a
step), to e4m3 by 2^-4 or, below its smallest normal number, half of 2^-9.
The fp32 statistics are sums of at most 16384 terms: a relative error far
below 2^-15, which is what the remaining terms allow.
"""
import ctypes

import pytest
import torch

from vision_transformer_shifted_gb300 import binding as sw

DEV = "cuda"
BF, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
FP = 2.0 ** -15
EPS = 1e-6


def reference(x, residual, gamma, eps=EPS):
    """s (bf16) and y (float64) of the definition."""
    s = x if residual is None else (x.float() + residual.float()).to(BF)
    d = s.double()
    return s, d / (d.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gamma.double()


def gradients(s, gamma, dy, dsum, eps=EPS):
    """dx, dgamma in float64 and the magnitudes their roundings go by."""
    s, gamma, dy = s.double(), gamma.double(), dy.double()
    r = (s.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n, a = s * r, dy * gamma
    m = (a * n).mean(-1, keepdim=True)
    dx = r * (a - n * m)
    size = r * (a.abs() + n.abs() * (a * n).abs().mean(-1, keepdim=True))
    if dsum is not None:
        dx, size = dx + dsum.double(), size + dsum.double().abs()
    return dx, (dy * n).sum(0), size, (dy * n).abs().sum(0)


def inputs(rows, C, residual=True, seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + rows * 4099 + C)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return ((n(rows, C) * 2).to(BF), n(rows, C).to(BF) if residual else None, (1 + 0.2 * n(C)).to(BF),
            n(rows, C).to(BF))


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


class rms:
    def __init__(self, C, eps=EPS):
        self.args = C, eps

    def __enter__(self):
        self.h = sw.swin_block_rms_create(*self.args)
        return self.h

    def __exit__(self, *exc):
        sw.swin_block_rms_destroy(self.h)


def close(got, ref, tol):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got.double()).all()
    assert (err <= tol).all(), float((err - tol).max())


# ---- CPU ---------------------------------------------------------------------------

@pytest.mark.parametrize("C,eps", [(0, 1e-6), (-8, 1e-6), (12, 1e-6), (16392, 1e-6), (64, -1e-6),
                                   (64, float("nan")), (64, float("inf"))])
def test_create_refuses(C, eps):
    h = ctypes.c_void_p(1)
    assert sw.load().swin_block_rms_create(ctypes.byref(h), C, eps) == sw.EINVAL
    assert h.value is None
    assert sw.load().swin_block_rms_create(None, 64, 1e-6) == sw.EINVAL


P = 1 << 20   # addresses that no refused call reads


def test_forward_refuses():
    lib = sw.load()
    n = 4 * 64 * 2   # bytes of a [4, 64] bf16 tensor
    ok = dict(x=P, residual=P + 4 * n, rows=4, gamma=P + 8 * n, out_sum=P + 12 * n, out=P + 16 * n)

    def call(**kw):
        a = {**ok, **kw}
        with rms(64) as h:
            rc = lib.swin_block_rms_forward(a.get("h", h), a["x"], a["residual"], a["rows"], a["gamma"],
                                            a["out_sum"], a["out"], None)
            rc8 = lib.swin_block_rms_forward_q8(a.get("h", h), a["x"], a["residual"], a["rows"], a["gamma"],
                                                a["out_sum"], a["out"], P + 32 * n, None)
        assert rc == rc8
        return rc

    assert call(rows=0) == sw.OK
    for bad in (dict(h=None), dict(x=None), dict(gamma=None), dict(out=None), dict(rows=-1), dict(x=P + 8),
                dict(residual=P + 4 * n + 2), dict(gamma=P + 8), dict(out=P + 16 * n + 4), dict(out_sum=P + 8),
                dict(residual=None), dict(out=P + 16), dict(out=ok["residual"] + 16), dict(out=ok["out_sum"]),
                dict(out_sum=P + 16), dict(out=ok["gamma"]), dict(out_sum=ok["gamma"])):
        assert call(**bad) == sw.EINVAL, bad
    with rms(64) as h:
        f = lib.swin_block_rms_forward_q8
        args = [h, P, None, 4, ok["gamma"], None]
        assert f(*args, ok["out"], None, None) == sw.EINVAL        # scales
        assert f(*args, ok["out"], P + 4, None) == sw.EINVAL       # misaligned scales
        assert f(*args, P, ok["out"], None) == sw.EINVAL           # codes over x
        assert f(*args, ok["out"], P, None) == sw.EINVAL           # scales over x
        assert f(*args, ok["out"], ok["out"], None) == sw.EINVAL   # scales over the codes


def test_backward_refuses():
    lib = sw.load()
    n = 4 * 64 * 2
    ok = dict(s=P, rows=4, gamma=P + 4 * n, dy=P + 8 * n, dsum=P + 12 * n, dx=P + 16 * n, dgamma=P + 20 * n)
    with rms(64) as h:
        for bad in (dict(h=None), dict(s=None), dict(gamma=None), dict(dy=None), dict(dx=None), dict(dgamma=None),
                    dict(rows=-1), dict(s=P + 8), dict(dsum=P + 8), dict(dgamma=P + 4), dict(dx=P), dict(dx=P + 16),
                    dict(dx=ok["dy"] + 16), dict(dx=ok["dsum"] + 16), dict(dx=ok["gamma"]), dict(dgamma=ok["s"]),
                    dict(dgamma=ok["dx"]), dict(dgamma=ok["gamma"])):
            a = {**ok, **bad}
            assert lib.swin_block_rms_backward(a.get("h", h), a["s"], a["rows"], a["gamma"], a["dy"], a["dsum"],
                                               a["dx"], a["dgamma"], None) == sw.EINVAL, bad
    assert lib.swin_block_rms_destroy(None) == sw.OK
    assert lib.swin_block_rms_last_launches(None) == 0


def test_binding_refuses_other_types_shapes_and_devices():
    x, r, g, _ = inputs(4, 64)
    with rms(64) as h:
        for kw in (dict(x=x.float()), dict(gamma=g[:32]), dict(residual=r[:2]), dict(x=x.t().contiguous().t()),
                   dict()):   # (the last: on the CPU)
            a = {**dict(x=x, gamma=g, residual=r), **kw}
            with pytest.raises(ValueError):
                sw.swin_block_rms_forward(h, a["x"], a["gamma"], torch.empty(4, 64, dtype=BF), residual=a["residual"])


def test_gradient_formula_against_differences():
    g = torch.Generator().manual_seed(3)
    s, gamma, dy, dsum = (torch.randn(*k, generator=g, dtype=torch.float64) for k in ((3, 8), (8,), (3, 8), (3, 8)))

    def loss(s, gamma):
        return float((s / (s.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * gamma * dy).sum() + (s * dsum).sum())

    dx, dgamma, _, _ = gradients(s, gamma, dy, dsum)
    for t, d in ((s, dx), (gamma, dgamma)):
        for i in range(t.numel()):
            e = torch.zeros(t.numel(), dtype=torch.float64)
            e[i] = 1e-5
            e = e.view(t.shape)
            diff = (loss(*((s + e, gamma) if t is s else (s, gamma + e)))
                    - loss(*((s - e, gamma) if t is s else (s, gamma - e)))) / 2e-5
            assert abs(diff - float(d.reshape(-1)[i])) < 1e-7


# ---- GPU ---------------------------------------------------------------------------

SHAPES = [(1, 8), (1, 2048), (3, 16), (33, 40), (257, 96), (70, 192), (19, 520), (9, 1016), (5, 1024), (7, 1032),
          (4, 2744), (3, 4096), (2, 8200), (2, 16384), (10007, 96)]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("residual", [True, False])
def test_forward(rows, C, residual):
    x, r, g, _ = inputs(rows, C, residual)
    s, y = reference(x, r, g)
    xd, rd, gd = dev(x, r, g)
    out = torch.full_like(xd, float("nan"))
    out_sum = torch.full_like(xd, float("nan")) if residual else None
    with rms(C) as h:
        sw.swin_block_rms_forward(h, xd, gd, out, residual=rd, out_sum=out_sum)
        assert sw.swin_block_rms_last_launches(h) == 1
    close(out, y, (2.0 ** -8 + FP) * y.abs())
    if residual:
        assert torch.equal(out_sum.cpu(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
def test_forward_q8(rows, C):
    residual = C % 16 == 0
    x, r, g, _ = inputs(rows, C, residual, seed=1)
    s, y = reference(x, r, g)
    xd, rd, gd = dev(x, r, g)
    codes = torch.full((rows, C), 5.0, device=DEV).to(E4M3)
    scales = torch.full((rows,), float("nan"), device=DEV)
    out_sum = torch.empty_like(xd) if residual else None
    with rms(C) as h:
        sw.swin_block_rms_forward_q8(h, xd, gd, codes, scales, residual=rd, out_sum=out_sum)
    ref = y.abs().amax(-1) / 448
    close(scales, ref, FP * ref)
    got = codes.float().double().cpu() * scales.double().cpu()[:, None]
    close(got, y, (2.0 ** -4 + FP) * y.abs() + 2.0 ** -10 * ref[:, None])
    if residual:
        assert torch.equal(out_sum.cpu(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("with_dsum", [True, False])
def test_backward(rows, C, with_dsum):
    s, dsum, g, dy = inputs(rows, C, with_dsum, seed=2)
    dx, dgamma, size, gsize = gradients(s, g, dy, dsum)
    sd, md, gd, yd = dev(s, dsum, g, dy)
    gx, gg = torch.full_like(sd, float("nan")), torch.full((C,), float("nan"), device=DEV)
    with rms(C) as h:
        sw.swin_block_rms_backward(h, sd, gd, yd, gx, gg, dsum=md)
        assert sw.swin_block_rms_last_launches(h) in (1, 2)
        again = torch.empty_like(gg)
        sw.swin_block_rms_backward(h, sd, gd, yd, gx, again, dsum=md)
    close(gx, dx, 2.0 ** -8 * dx.abs() + FP * size)
    close(gg, dgamma, FP * gsize)
    assert torch.equal(gg, again)   # a fixed order of summation


@pytest.mark.gpu
def test_rows_past_32_bits_of_elements():
    """rows * C > 2^31: the last rows, which lie past 32-bit offsets."""
    C, rows = 16384, (1 << 17) + 5
    x = torch.zeros(rows, C, dtype=BF, device=DEV)
    tail, _, g, _ = inputs(7, C, False, seed=5)
    x[-7:] = tail.to(DEV)
    out = torch.empty_like(x)
    with rms(C) as h:
        sw.swin_block_rms_forward(h, x, g.to(DEV), out)
    _, y = reference(tail, None, g)
    close(out[-7:], y, (2.0 ** -8 + FP) * y.abs())
    assert not out[:-7].any()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 2744])
def test_in_place(C):
    x, r, g, dy = inputs(37, C, True, seed=3)
    s, y = reference(x, r, g)
    xd, rd, gd, yd = dev(x, r, g, dy)
    with rms(C) as h:
        sw.swin_block_rms_forward(h, xd, gd, xd, residual=rd, out_sum=rd)
        close(xd, y, (2.0 ** -8 + FP) * y.abs())
        assert torch.equal(rd.cpu(), s)
        dx, _, size, _ = gradients(s, g, dy, x)
        gg = torch.empty(C, device=DEV)
        one, two = yd.clone(), x.to(DEV)
        sw.swin_block_rms_backward(h, rd, gd, one, one, gg, dsum=two)
        close(one, dx, 2.0 ** -8 * dx.abs() + FP * size)
        sw.swin_block_rms_backward(h, rd, gd, yd, two, gg, dsum=two)
        assert torch.equal(one, two)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 2744])
def test_zero_infinite_and_nan_rows(C):
    x, _, g, _ = inputs(6, C, False, seed=4)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, C - 1] = float("nan")
    xd, gd = dev(x, g)
    out, codes, scales = torch.empty_like(xd), torch.empty(6, C, dtype=E4M3, device=DEV), torch.empty(6, device=DEV)
    with rms(C) as h:
        sw.swin_block_rms_forward(h, xd, gd, out)
        sw.swin_block_rms_forward_q8(h, xd, gd, codes, scales)
    q = codes.float().cpu()
    assert not out[1].any() and not q[1].any() and 0 < float(scales[1]) < 1e-30
    assert out[3].isnan().all() and q[2:4].isnan().all() and scales[2:4].isnan().all()
    assert out[2, 5].isnan() and not out[2, :5].any()   # an infinity makes r zero
    good = [0, 4, 5]
    _, y = reference(x[good], None, g)
    close(out[good], y, (2.0 ** -8 + FP) * y.abs())
    close(q[good] * scales.cpu()[good][:, None], y,
          (2.0 ** -4 + FP) * y.abs() + 2.0 ** -10 * y.abs().amax(-1, keepdim=True) / 448)


@pytest.mark.gpu
def test_empty_batch():
    C = 96
    x = torch.empty(0, C, dtype=BF, device=DEV)
    g, gg = torch.ones(C, dtype=BF, device=DEV), torch.full((C,), 3.0, device=DEV)
    with rms(C) as h:
        sw.swin_block_rms_forward(h, x, g, x.clone())
        sw.swin_block_rms_backward(h, x, g, x.clone(), x.clone(), gg)
    assert not gg.any()


@pytest.mark.gpu
def test_rows_behind_the_batch_stay():
    C, rows = 192, 45
    x, r, g, dy = dev(*inputs(64, C, True, seed=6))
    out, out_sum, dx = (torch.full_like(x, 7.0) for _ in range(3))
    codes, scales = torch.full((64, C), 7.0, device=DEV).to(E4M3), torch.full((64,), 7.0, device=DEV)
    with rms(C) as h:
        sw.swin_block_rms_forward(h, x[:rows], g, out[:rows], residual=r[:rows], out_sum=out_sum[:rows])
        sw.swin_block_rms_forward_q8(h, x[:rows], g, codes[:rows], scales[:rows])
        sw.swin_block_rms_backward(h, x[:rows], g, dy[:rows], dx[:rows], torch.empty(C, device=DEV))
    for t in (out, out_sum, dx, codes.float(), scales):
        assert (t[rows:] == 7).all() and not (t[:rows] == 7).all()


@pytest.mark.gpu
def test_streams_and_captured_graphs_share_nothing():
    """One handle: eager calls on two streams at once and two captured graphs,
    replayed on new inputs while eager calls run, give the eager results."""
    C, rows = 2048, 3000
    s, _, g, dy = dev(*inputs(rows, C, False, seed=7))
    s2, _, _, dy2 = dev(*inputs(rows, C, False, seed=8))
    with rms(C) as h:
        def call(s, dy):
            dx, gg = torch.empty_like(s), torch.empty(C, device=DEV)
            sw.swin_block_rms_backward(h, s, g, dy, dx, gg)
            return dx, gg

        want, want2 = call(s, dy), call(s2, dy2)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for k in range(6):
            with torch.cuda.stream(streams[k % 2]):
                got.append(call(*((s, dy) if k % 2 else (s2, dy2))))
        torch.cuda.synchronize()
        for k, o in enumerate(got):
            w = want if k % 2 else want2
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
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
            assert torch.equal(o[0], want2[0]) and torch.equal(o[1], want2[1])
        assert torch.equal(eager[0], want[0]) and torch.equal(eager[1], want[1])


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
    with rms(8) as h, pytest.raises(ValueError, match="rows"):
        sw.swin_block_rms_forward(h, Tall(), None, None)


@pytest.mark.gpu
def test_two_host_threads_with_a_handle_each():
    """Handles of different widths used from two threads at once: what one call
    asks of a kernel (its shared memory) does not take from the other's."""
    import threading
    failures = []

    def work(C, rows):
        try:
            s, _, g, dy = dev(*inputs(rows, C, False, seed=C))
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with rms(C) as h, torch.cuda.stream(stream):
                dx, dg = torch.empty_like(s), torch.empty(C, device=DEV)
                for _ in range(400):
                    sw.swin_block_rms_backward(h, s, g, dy, dx, dg)
                stream.synchronize()
        except Exception as e:
            failures.append((C, e))

    threads = [threading.Thread(target=work, args=a) for a in ((1000, 8), (16384, 8), (10000, 3))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures, failures


@pytest.mark.gpu
@pytest.mark.parametrize("C", [8, 96, 192, 768, 2744])
@pytest.mark.parametrize("rows", [1, 3, 300, 5003])
@pytest.mark.parametrize("with_dsum", [True, False])
def test_backward_without_eps(rows, C, with_dsum):
    """eps = 0 and no row of zeros: every gradient is finite, whatever part of a
    block the rows leave empty (there the mean of the squares is zero, and one
    over its root infinite)."""
    s, dsum, g, dy = inputs(rows, C, with_dsum, seed=9)
    dx, dgamma, size, gsize = gradients(s, g, dy, dsum, eps=0.0)
    sd, md, gd, yd = dev(s, dsum, g, dy)
    gx, gg = torch.full_like(sd, float("nan")), torch.full((C,), float("nan"), device=DEV)
    with rms(C, 0.0) as h:
        sw.swin_block_rms_backward(h, sd, gd, yd, gx, gg, dsum=md)
    close(gx, dx, 2.0 ** -8 * dx.abs() + FP * size)
    close(gg, dgamma, FP * gsize)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [512, 4096])
@pytest.mark.parametrize("amax", [1.53125, 1.078125, 1.625, 1.75])
def test_codes_are_the_rounded_quotients(C, amax):
    """Rows of +-1 with eps = 0: r is 1 and y = s gamma exactly, so that code and
    scale are known to the last bit.  gamma holds every bf16 value of four
    octaves up to amax; some of their quotients lie on the middle between two
    codes, where y times 1 / scale rounds to the other one."""
    v = torch.arange(0x3e00, 0x4000, dtype=torch.int32).to(torch.int16).view(BF)   # 0.125 to 2
    v = v[v.float() <= amax]
    gamma = torch.full((C,), amax, dtype=BF)
    gamma[:v.numel()] = v
    sign = torch.randint(0, 2, (9, C), generator=torch.Generator().manual_seed(C)) * 2 - 1
    x = sign.to(BF)
    xd, gd = dev(x, gamma)
    codes, scales = torch.empty(9, C, dtype=E4M3, device=DEV), torch.empty(9, device=DEV)
    with rms(C, 0.0) as h:
        sw.swin_block_rms_forward_q8(h, xd, gd, codes, scales)
    scale = torch.tensor(amax) / 448
    assert (scales.cpu() == scale).all()
    assert torch.equal(codes.cpu().float(), (x.float() * gamma.float() / scale).to(E4M3).float())


@pytest.mark.gpu
def test_codes_of_products_are_the_rounded_quotients():
    """The same with y of 16 bits: rows of multiples of 1/128 whose mean square is
    one (eight squares of whole numbers with the sum 8 * 128^2, time and again),
    where the sums are exact and r is 1."""
    import random
    rng = random.Random(5)
    C, rows, squares = 512, 400, {i * i: i for i in range(1, 256)}

    def eight():
        while True:
            v = [rng.randint(1, 200) for _ in range(7)]
            left = 8 * 128 * 128 - sum(i * i for i in v)
            if left in squares:
                return v + [squares[left]]

    some = [eight() for _ in range(300)]
    x = torch.tensor([[i * rng.choice((-1, 1)) for _ in range(C // 8) for i in rng.choice(some)]
                      for _ in range(rows)]).double().div(128).to(BF)
    assert (x.double().pow(2).mean(-1) == 1).all()
    gamma = (1 + 0.2 * torch.randn(C, generator=torch.Generator().manual_seed(6))).to(BF)
    y = x.float() * gamma.float()
    scale = y.abs().amax(-1) / 448
    want = (y / scale[:, None]).to(E4M3).float()
    assert not torch.equal(want, (y * (1 / scale)[:, None]).to(E4M3).float())
    codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.empty(rows, device=DEV)
    with rms(C, 0.0) as h:
        sw.swin_block_rms_forward_q8(h, *dev(x, gamma), codes, scales)
    assert torch.equal(scales.cpu(), scale)
    assert torch.equal(codes.cpu().float(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("factor", [2.0 ** -120, 2.0 ** -95, 2.0 ** -60, 2.0 ** 100, float("inf")])
def test_codes_of_very_small_and_large_rows(factor):
    """y from gamma (x of +-1, eps = 0) down to where a row's scale stands at its
    floor, up to 2^101, and infinite."""
    C = 256
    gamma = torch.randn(C, generator=torch.Generator().manual_seed(7)).to(BF)
    if factor == float("inf"):
        gamma[3] = factor
    else:
        gamma = (gamma.float() * factor).to(BF)
    x = torch.ones(3, C, dtype=BF)
    x[1] = -1
    codes, scales = torch.empty(3, C, dtype=E4M3, device=DEV), torch.empty(3, device=DEV)
    with rms(C, 0.0) as h:
        sw.swin_block_rms_forward_q8(h, *dev(x, gamma), codes, scales)
    scale = gamma.float().abs().amax().clamp_min(1e-30) / 448
    assert (scales.cpu() == scale).all()
    want = (x.float() * gamma.float() / scale).to(E4M3).float()
    assert torch.equal(codes.cpu().float().nan_to_num(nan=7e7), want.nan_to_num(nan=7e7))


@pytest.mark.gpu
def test_backward_and_codes_past_32_bits_of_elements():
    """rows * C > 2^31: rows at the beginning, around the 2^31st element and at the
    end; dgamma over all of them.  Its sums in fp32: some 863 rows a block one
    after the other and 152 partial rows, each addition off by 2^-24 at most."""
    C, rows = 16384, (1 << 17) + 5
    gen = torch.Generator(device=DEV).manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV, dtype=BF)  # noqa: E731
    s, dy, g = n(rows, C), n(rows, C), 1 + 0.2 * n(C)
    dx, dgamma = torch.full_like(s, float("nan")), torch.full((C,), float("nan"), device=DEV)
    codes, scales = torch.empty(rows, C, dtype=E4M3, device=DEV), torch.full((rows,), float("nan"), device=DEV)
    with rms(C) as h:
        sw.swin_block_rms_backward(h, s, g, dy, dx, dgamma)
        sw.swin_block_rms_forward_q8(h, s, g, codes, scales)
    some = [0, 1, 65535, 131070, 131071, 131072, 131073, rows - 1]
    ref, _, size, _ = gradients(s[some].cpu(), g.cpu(), dy[some].cpu(), None)
    close(dx[some], ref, 2.0 ** -8 * ref.abs() + FP * size)
    _, y = reference(s[some].cpu(), None, g.cpu())
    scale = y.abs().amax(-1) / 448
    close(scales[some], scale, FP * scale)
    got = codes[some].float().double().cpu() * scales[some].double().cpu()[:, None]
    close(got, y, (2.0 ** -4 + FP) * y.abs() + 2.0 ** -10 * scale[:, None])
    ref, size = torch.zeros(C, dtype=torch.float64), torch.zeros(C, dtype=torch.float64)
    for i in range(0, rows, 8192):
        _, d, _, m = gradients(s[i:i + 8192], g, dy[i:i + 8192], None)
        ref += d.cpu()
        size += m.cpu()
    close(dgamma, ref, ((863 + 152) * 2.0 ** -24 + FP) * size)


@pytest.mark.gpu
def test_two_host_threads_compute_what_one_does():
    """A handle a thread at once: every result is the one that the call gives alone."""
    import threading
    wrong, data = [], []
    for C, rows in ((1000, 8), (16384, 8), (10000, 3), (96, 3001), (2744, 1500)):
        s, _, g, dy = dev(*inputs(rows, C, False, seed=C))
        dx, dg = torch.empty_like(s), torch.empty(C, device=DEV)
        with rms(C) as h:
            sw.swin_block_rms_backward(h, s, g, dy, dx, dg)
        data.append((C, s, g, dy, dx, dg))
    torch.cuda.synchronize()

    def work(C, s, g, dy, dx, dg):
        try:
            stream = torch.cuda.Stream()
            with rms(C) as h, torch.cuda.stream(stream):
                for _ in range(100):
                    one, two = torch.empty_like(dx), torch.empty_like(dg)
                    sw.swin_block_rms_backward(h, s, g, dy, one, two)
                    stream.synchronize()
                    if not (torch.equal(one, dx) and torch.equal(two, dg)):
                        wrong.append(C)
        except Exception as e:
            wrong.append((C, e))

    threads = [threading.Thread(target=work, args=a) for a in data]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
