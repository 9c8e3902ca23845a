"""GPU tests of the row operators (norm, its backward, 8-bit rows, the 8-bit
UVQK projection) against their formulas in 64 bits.

Tolerances count the roundings: half a step of the output's type relative to
the value (bf16 2^-8, fp32 2^-24, e4m3 2^-4 and half of its smallest step,
2^-10, near zero), and fp32 sums of n terms to n 2^-24 of the sum of their
magnitudes.
"""
import pytest
import torch

import pointwise_attention_b200 as pa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
EPS = 1e-6
U = 2.0 ** -24


def rows(seed, T, E, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(T, E, generator=g)).to(dtype).to(DEV)


def within(got, ref, tol, what):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, what
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() - tol
    assert bool((bad <= 0).all()), "%s: off by %.3e over %.3e" % (
        what, float((got - ref).abs().max()), float(bad.max()))


def norm64(x, res, w, dtype):
    h = x if res is None else (x.double() + res.double()).to(dtype)
    hd = h.double()
    r = 1.0 / torch.sqrt((hd * hd).mean(1) + EPS)
    v = hd * r[:, None]
    return h, r, v if w is None else v * w.double()


def check_q8(q8, scale, v, E, what):
    top = v.abs().amax(1).clamp_min(2.0 ** -100)
    rel = (E + 16) * U
    within(scale, top / 448.0, rel * top / 448.0, what + " scale")
    # half a step of e4m3 relative to the value, at least half its smallest
    # step; the value before the rounding is off by fp32's share
    s = scale.double()[:, None]
    within(q8.double() * s, v, v.abs() * (2.0 ** -4 + 3 * rel) + s * 2.0 ** -10 * (1 + rel), what)


SHAPES = [(1, 1), (1, 16), (3, 7), (5, 256), (17, 512), (9, 513), (8, 1000), (33, 1024), (6, 1032),
          (4, 2048), (3, 2055), (2, 4096), (3, 5000), (2, 8192), (2, 8200), (2, 16384), (1, 16383),
          (1025, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", SHAPES)
def test_norm_forward(T, E, dtype):
    x, res = rows(T + E, T, E, dtype), rows(T + E + 1, T, E, dtype)
    w = (1.0 + 0.3 * rows(3, 1, E, F32)[0])
    rel = (E + 16) * U
    for r_, w_ in ((res, w), (None, w), (res, None)):
        h, rstd, v = norm64(x, r_, w_, dtype)
        out = pa.hstu_rmsnorm_fwd(x, residual=r_, weight=w_, eps=EPS, save_rstd=True)
        if r_ is None:
            assert out["h"] is None
        else:
            assert torch.equal(out["h"], h)
        assert out["q8"] is None
        within(out["rstd"], rstd, rel * rstd, "rstd")
        within(out["y"], v, v.abs() * (HALF[dtype] + 2 * rel), "y")
        q = pa.hstu_rmsnorm_fwd(x, residual=r_, weight=w_, eps=EPS, quant=True)
        assert q["y"] is None and q["rstd"] is None
        check_q8(q["q8"], q["scale"], v, E, "q8")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", SHAPES)
def test_norm_backward(T, E, dtype):
    h, dy, dres = (rows(s + E, T, E, dtype) for s in (1, 2, 3))
    w = 1.0 + 0.3 * rows(3, 1, E, F32)[0]
    rstd = (1.0 / torch.sqrt((h.double() ** 2).mean(1) + EPS)).float()
    hd, dyd, r = h.double(), dy.double(), rstd.double()[:, None]
    for w_, d_ in ((w, dres), (w, None), (None, dres)):
        g = dyd if w_ is None else dyd * w_.double()
        m = (g * hd).mean(1, keepdim=True)
        dx = r * (g - hd * r * r * m)
        dw = (dyd * hd * r).sum(0)
        rel = (E + 16) * U
        mabs = (g * hd).abs().mean(1, keepdim=True)
        tol = r * (g.abs() * 4 * U + hd.abs() * r * r * mabs * rel)
        if d_ is not None:
            dx = dx + d_.double()
            tol = tol + d_.double().abs() * 2 * U
        got, gw = pa.hstu_rmsnorm_bwd(dy, h, rstd, weight=w_, d_residual=d_)
        within(got, dx, tol + dx.abs() * (HALF[dtype] + 2 * U), "dx")
        within(gw, dw, (dyd * hd * r).abs().sum(0) * (T + 8) * U, "dw")
        got2, none = pa.hstu_rmsnorm_bwd(dy, h, rstd, weight=w_, d_residual=d_,
                                         need_weight_grad=False)
        assert none is None and torch.equal(got, got2)


def test_norm_backward_against_differences():
    """The gradients are those of the forward: central differences in 64 bits
    of L = sum(y c) + sum(h e)."""
    T, E = 3, 40
    x, res, c, e = (rows(s, T, E, F32) for s in (1, 2, 3, 4))
    w = 1.0 + 0.3 * rows(5, 1, E, F32)[0]
    out = pa.hstu_rmsnorm_fwd(x, residual=res, weight=w, eps=EPS, save_rstd=True)
    dx, dw = pa.hstu_rmsnorm_bwd(c, out["h"], out["rstd"], weight=w, d_residual=e)

    def loss(xd, wd):
        h = xd + res.double()
        v = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * wd
        return float((v * c.double()).sum() + (h * e.double()).sum())

    step = 1e-4   # differences are off by step^2 times third derivatives of order ten
    for t, i in ((0, 0), (1, 17), (2, 39)):
        d = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        d[t, i] = step
        num = (loss(x.double() + d, w.double()) - loss(x.double() - d, w.double())) / (2 * step)
        assert abs(num - float(dx[t, i])) <= 1e-6 + 1e-5 * abs(num)
    for i in (0, 21, 39):
        d = torch.zeros(E, dtype=torch.float64, device=DEV)
        d[i] = step
        num = (loss(x.double(), w.double() + d) - loss(x.double(), w.double() - d)) / (2 * step)
        assert abs(num - float(dw[i])) <= 1e-6 + 1e-5 * abs(num)


def test_norm_backward_many_rows_repeats_bitwise():
    """More rows than blocks: each block walks several; the sums' order is fixed."""
    T, E = 5003, 96
    h, dy = rows(1, T, E, BF16), rows(2, T, E, BF16)
    rstd = (1.0 / torch.sqrt((h.double() ** 2).mean(1) + EPS)).float()
    dx, dw = pa.hstu_rmsnorm_bwd(dy, h, rstd)
    terms = dy.double() * h.double() * rstd.double()[:, None]
    within(dw, terms.sum(0), terms.abs().sum(0) * (T + 8) * U, "dw")
    dx2, dw2 = pa.hstu_rmsnorm_bwd(dy, h, rstd)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def check_many_rows(T, E, dtype):
    x, res, dy = (rows(s, T, E, dtype) for s in (1, 2, 3))
    rel = (E + 16) * U
    h, rstd, v = norm64(x, res, None, dtype)
    out = pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, save_rstd=True)
    assert torch.equal(out["h"], h)
    within(out["rstd"], rstd, rel * rstd, "rstd")
    within(out["y"], v, v.abs() * (HALF[dtype] + 2 * rel), "y")
    q8, s = pa.hstu_quant_rows(x)
    check_q8(q8, s, x.double(), E, "q8")
    dx, dw = pa.hstu_rmsnorm_bwd(dy, h, out["rstd"], d_residual=res)
    hd, dyd, r = h.double(), dy.double(), out["rstd"].double()[:, None]
    m, mabs = (dyd * hd).mean(1, keepdim=True), (dyd * hd).abs().mean(1, keepdim=True)
    ref = r * (dyd - hd * r * r * m) + res.double()
    tol = r * (dyd.abs() * 4 * U + hd.abs() * r * r * mabs * rel) + res.double().abs() * 2 * U
    within(dx, ref, tol + ref.abs() * (HALF[dtype] + 2 * U), "dx")
    terms = dyd * hd * r
    within(dw, terms.sum(0), terms.abs().sum(0) * (T + 8) * U, "dw")


@pytest.mark.parametrize("dtype,E", [(BF16, 24), (F32, 20), (BF16, 520), (F32, 7)])
def test_many_rows_a_warp(dtype, E):
    """Every warp walks several rows (more than are under way at a time)."""
    check_many_rows(50021 if E < 500 else 30011, E, dtype)


@pytest.mark.parametrize("T,E,dtype", [
    (200003, 8, BF16), (150001, 64, BF16), (150001, 16, F32), (100003, 40, F32), (60001, 33, BF16),
    (60001, 128, BF16), (60001, 65, F32), (50021, 256, BF16), (20011, 301, F32), (20011, 301, BF16),
    (4801, 2048, BF16), (4801, 2048, F32), (4801, 4096, BF16), (4801, 4096, F32),
    (4801, 8192, BF16), (4801, 8000, F32), (2411, 8001, F32), (2411, 16384, BF16)])
def test_many_rows_of_every_shape(T, E, dtype):
    check_many_rows(T, E, dtype)


NARROW = [(1, 3), (2, 16), (3, 30), (5, 32), (515, 32), (37, 50), (9, 64), (70, 100), (13, 128),
          (6, 136), (9, 200), (7, 300), (9, 333), (2, 2001), (2, 4001)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", NARROW)
def test_rows_narrower_than_a_warp(T, E, dtype):
    test_norm_forward(T, E, dtype)
    test_norm_backward(T, E, dtype)
    test_quant_rows(T, E, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", [(1, 2), (9, 22), (5, 66), (5, 130), (3, 258), (9, 514), (3, 1030),
                                 (2, 2050), (2, 4098), (2, 8194), (1, 16382)])
def test_rows_of_even_length(T, E, dtype):
    test_norm_forward(T, E, dtype)
    test_norm_backward(T, E, dtype)
    test_quant_rows(T, E, dtype)


@pytest.mark.parametrize("T,E", [(100003, 30), (60001, 100), (50021, 202), (20011, 500),
                                 (9001, 1002), (4801, 2004), (4801, 4002), (2411, 8002)])
def test_many_rows_of_even_length(T, E):
    check_many_rows(T, E, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_rows_off_their_vectors(dtype, off):
    """Rows that start `off` elements past a 16-byte boundary, and a weight that
    does: the same results to the rounding's order of sums, bit for bit in h."""
    T, E = 37, 64
    def shift(t):
        b = t.new_zeros(t.numel() + 8)
        b[off:off + t.numel()] = t.flatten()
        return b[off:off + t.numel()].view(t.shape)
    x, res, dy = (shift(rows(s, T, E, dtype)) for s in (1, 2, 3))
    w = shift(1.0 + 0.3 * rows(4, 1, E, F32)[0])
    rel = (E + 16) * U
    h, rstd, v = norm64(x, res, w, dtype)
    out = pa.hstu_rmsnorm_fwd(x, residual=res, weight=w, eps=EPS, save_rstd=True)
    assert torch.equal(out["h"], h)
    within(out["y"], v, v.abs() * (HALF[dtype] + 2 * rel), "y")
    q8, s = pa.hstu_quant_rows(x)
    check_q8(q8, s, x.double(), E, "q8")
    dx, dw = pa.hstu_rmsnorm_bwd(dy, h, out["rstd"], weight=w)
    dx2, dw2 = pa.hstu_rmsnorm_bwd(dy.clone(), h.clone(), out["rstd"], weight=w.clone())
    terms = dy.double() * h.double() * out["rstd"].double()[:, None]
    within(dw, terms.sum(0), terms.abs().sum(0) * (T + 8) * U, "dw")
    g, hd, r = dy.double() * w.double(), h.double(), out["rstd"].double()[:, None]
    m, mabs = (g * hd).mean(1, keepdim=True), (g * hd).abs().mean(1, keepdim=True)
    ref = r * (g - hd * r * r * m)
    tol = r * (g.abs() * 4 * U + hd.abs() * r * r * mabs * rel) + ref.abs() * (HALF[dtype] + 2 * U)
    within(dx, ref, tol, "dx")
    within(dx2, ref, tol, "dx")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", [(1, 16), (5, 32), (3, 64), (7, 128), (2, 50), (1, 512), (33, 24)])
def test_rows_behind_the_last_stay(T, E, dtype):
    """Rows and values past T of larger tensors hold NaN, which nothing reads,
    and stay: a warp's rows may end inside it."""
    R = T + 70
    big = [rows(s, R, E, dtype) for s in (1, 2, 3)]
    for t in big:
        t[T:] = float("nan")
    x, res, dy = (t[:T] for t in big)
    outs = {k: torch.full((R, E), 7.0, dtype=dtype, device=DEV) for k in ("h", "y")}
    outs["rstd"] = torch.full((R,), 7.0, device=DEV)
    out = pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, save_rstd=True,
                              out={k: t[:T] for k, t in outs.items()})
    h, _, v = norm64(x, res, None, dtype)
    assert torch.equal(out["h"], h)
    within(out["y"], v, v.abs() * (HALF[dtype] + 2 * (E + 16) * U), "y")
    for t in outs.values():
        assert bool((t[T:] == 7.0).all())
    q8 = {"q8": torch.zeros(R, E, dtype=torch.float8_e4m3fn, device=DEV),
          "scale": torch.full((R,), 7.0, device=DEV)}
    pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, quant=True, out={k: t[:T] for k, t in q8.items()})
    assert bool((q8["scale"][T:] == 7.0).all()) and bool((q8["q8"][T:].float() == 0).all())
    dx = torch.full((R, E), 7.0, dtype=dtype, device=DEV)
    _, dw = pa.hstu_rmsnorm_bwd(dy, out["h"], out["rstd"], d_residual=res, dx=dx[:T])
    assert bool((dx[T:] == 7.0).all()) and bool(torch.isfinite(dx).all())
    terms = dy.double() * h.double() * out["rstd"].double()[:, None]
    within(dw, terms.sum(0), terms.abs().sum(0) * (T + 8) * U, "dw")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E", SHAPES)
def test_quant_rows(T, E, dtype):
    x = rows(T * E, T, E, dtype)
    q8, s = pa.hstu_quant_rows(x)
    check_q8(q8, s, x.double(), E, "q8")


def test_unaligned_rows_and_no_rows():
    base = rows(1, 1, 6 * 64 + 1, BF16)[0]
    x = base[1:].view(6, 64)                 # 2-byte aligned
    out = pa.hstu_rmsnorm_fwd(x, eps=EPS)
    ref = pa.hstu_rmsnorm_fwd(x.clone(), eps=EPS)
    _, _, v = norm64(x, None, None, BF16)
    for o in (out, ref):
        within(o["y"], v, v.abs() * (HALF[BF16] + 200 * U), "y")
    empty = torch.empty(0, 64, dtype=BF16, device=DEV)
    assert pa.hstu_rmsnorm_fwd(empty)["y"].shape == (0, 64)
    dx, dw = pa.hstu_rmsnorm_bwd(empty, empty, torch.empty(0, device=DEV))
    assert dx.shape == (0, 64) and torch.equal(dw, torch.zeros(64, device=DEV))
    assert pa.hstu_quant_rows(empty)[0].shape == (0, 64)


def test_zero_rows_nan_rows_and_neighbours():
    x = rows(1, 8, 128, BF16)
    x[2] = 0.0
    x[4, 100] = float("nan")
    x[6, 3] = float("inf")
    y = pa.hstu_rmsnorm_fwd(x, eps=EPS)["y"]
    q = pa.hstu_rmsnorm_fwd(x, eps=EPS, quant=True)
    assert torch.equal(y[2], torch.zeros_like(y[2])) and torch.isnan(y[4]).all()
    assert torch.equal(q["q8"][2].float(), torch.zeros(128, device=DEV))
    # the scale is the fp32 number nearest to 2^-100 / 448 (which is not one)
    assert q["scale"][2].cpu() == torch.tensor(2.0 ** -100 / 448, dtype=F32)
    assert torch.isnan(q["scale"][4])
    for t in (0, 1, 3, 5, 7):
        _, _, v = norm64(x[t:t + 1], None, None, BF16)
        within(y[t:t + 1], v, v.abs() * (HALF[BF16] + 300 * U), "y")


def test_outputs_over_inputs():
    """The residual stream updated in place; dx over d_residual."""
    x, res = rows(1, 77, 512, BF16), rows(2, 77, 512, BF16)
    want = pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, save_rstd=True)
    res2 = res.clone()
    got = pa.hstu_rmsnorm_fwd(x, residual=res2, eps=EPS, out=dict(h=res2))
    assert torch.equal(got["h"], want["h"]) and got["h"].data_ptr() == res2.data_ptr()
    assert torch.equal(got["y"], want["y"])
    dy, dres = rows(3, 77, 512, BF16), rows(4, 77, 512, BF16)
    dx, dw = pa.hstu_rmsnorm_bwd(dy, want["h"], want["rstd"], d_residual=dres)
    d2 = dres.clone()
    dx2, dw2 = pa.hstu_rmsnorm_bwd(dy, want["h"], want["rstd"], d_residual=d2, dx=d2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype,E", [(BF16, 512), (F32, 100), (F32, 33), (BF16, 2048)])
def test_more_outputs_over_inputs(dtype, E):
    """The stream over x, the norm over the residual; y and 8 bits from one
    call; dx over dy."""
    x, res = rows(1, 50, E, dtype), rows(2, 50, E, dtype)
    want = pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, save_rstd=True)
    q = pa.hstu_rmsnorm_fwd(x, residual=res, eps=EPS, quant=True)
    a, b = x.clone(), res.clone()
    got = pa.hstu_rmsnorm_fwd(a, residual=b, eps=EPS, quant=True, out=dict(h=a, y=b))
    assert torch.equal(got["h"], want["h"]) and got["h"].data_ptr() == a.data_ptr()
    assert torch.equal(got["y"], want["y"]) and got["y"].data_ptr() == b.data_ptr()
    assert torch.equal(got["q8"].float(), q["q8"].float()) and torch.equal(got["scale"], q["scale"])
    dy = rows(3, 50, E, dtype)
    dx, dw = pa.hstu_rmsnorm_bwd(dy, want["h"], want["rstd"], d_residual=res)
    d2 = dy.clone()
    dx2, dw2 = pa.hstu_rmsnorm_bwd(d2, want["h"], want["rstd"], d_residual=res, dx=d2)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_a_given_stream_and_wrong_arguments():
    x = rows(1, 40, 256, BF16)
    want = pa.hstu_rmsnorm_fwd(x, eps=EPS)["y"]
    s = torch.cuda.Stream()
    y = torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    pa.hstu_rmsnorm_fwd(x, eps=EPS, out=dict(y=y), stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    for bad in (lambda: pa.hstu_rmsnorm_fwd(x.t()), lambda: pa.hstu_rmsnorm_fwd(x[0]),
                lambda: pa.hstu_rmsnorm_fwd(x, residual=x.float()),
                lambda: pa.hstu_rmsnorm_fwd(x, weight=torch.ones(255, device=DEV)),
                lambda: pa.hstu_rmsnorm_fwd(x.half()),
                lambda: pa.hstu_rmsnorm_bwd(x, x, torch.ones(39, device=DEV)),
                lambda: pa.hstu_quant_rows(x[:, :128])):
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------ 8-bit projection
def silu64(x):
    return x / (1.0 + torch.exp(-x))


def project(seed, T, E, H, dqk, dv, act, bias, what):
    N = 2 * H * (dqk + dv)
    x8, xs = pa.hstu_quant_rows(rows(seed, T, E, F32))
    w8, ws = pa.hstu_quant_rows(rows(seed + 1, N, E, F32, std=E ** -0.5))
    b = 0.2 * rows(seed + 2, 1, N, F32)[0] if bias else None
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = pa.hstu_uvqk_fp8_fwd(x8, xs, w8, ws, H, dqk, dv, bias=b, act=act, workspace=status)
    assert pa.hstu_attn_check(status) == 0
    xd, wd = x8.double() * xs.double()[:, None], w8.double() * ws.double()[:, None]
    p = xd @ wd.t()
    mag = xd.abs() @ wd.abs().t()
    if b is not None:
        p = p + b.double()
    # fp32 sums of E products, four roundings after them; SiLU's slope is at
    # most 1.1, and it is x/2 (1 + tanh(x/2)) with the hardware's tanh, whose
    # documented relative error is 2^-11: |x|/2 2^-11
    tol = mag * (E + 4) * U + p.abs() * 4 * U
    if act:
        p, tol = silu64(p), 1.1 * tol + p.abs() * 2.0 ** -12
    tol = tol + p.abs() * HALF[BF16] + 1e-30
    at = 0
    for n, w_ in (("u", dv), ("v", dv), ("q", dqk), ("k", dqk)):
        got = out[n].reshape(T, -1)
        within(got, p[:, at:at + H * w_], tol[:, at:at + H * w_], what + " " + n)
        at += H * w_
    return out


@pytest.mark.parametrize("T", [1, 17, 128, 129, 300])
@pytest.mark.parametrize("E,H,dqk,dv,act,bias", [
    (16, 2, 128, 128, 1, True), (64, 2, 128, 128, 0, False), (80, 4, 64, 128, 1, True),
    (512, 4, 128, 128, 1, True), (528, 8, 128, 128, 0, True), (1040, 2, 128, 128, 1, False),
    (256, 1, 256, 512, 1, True)])
def test_uvqk_fp8(T, E, H, dqk, dv, act, bias):
    project(T + E, T, E, H, dqk, dv, act, bias, "uvqk")


@pytest.mark.parametrize("T,E", [(1111, 192), (1250, 192), (5000, 192), (40001, 192), (1300, 1024),
                                 (5000, 1024), (3000, 1536)])
def test_uvqk_fp8_many_rows(T, E):
    project(T, T, E, 4, 128, 128, 1, True, "uvqk")


def test_uvqk_fp8_outputs_stay_inside(monkeypatch):
    """Rows behind the last token and unaligned-by-32 outputs: nothing else is
    written."""
    T, E, H = 70, 128, 2
    x8, xs = pa.hstu_quant_rows(rows(1, T, E, F32))
    w8, ws = pa.hstu_quant_rows(rows(2, 1024, E, F32))
    ref = pa.hstu_uvqk_fp8_fwd(x8, xs, w8, ws, H, 128, 128, act=1)
    big = {n: torch.full((T * 256 + 256 + 8,), 7.0, dtype=BF16, device=DEV) for n in "uvqk"}
    out = {n: big[n][8:8 + T * 256].view((T, 256) if n == "u" else (T, 2, 128)) for n in "uvqk"}
    pa.hstu_uvqk_fp8_fwd(x8, xs, w8, ws, H, 128, 128, act=1, out=out)
    for n in "uvqk":
        assert torch.equal(out[n], ref[n])
        assert bool((big[n][:8] == 7).all()) and bool((big[n][8 + T * 256:] == 7).all())


def test_capture_and_other_stream():
    """Norm to 8 bits and projection captured in one graph, replayed on new
    inputs on a side stream."""
    T, E, H = 200, 256, 2
    x = rows(1, T, E, BF16)
    w8, ws = pa.hstu_quant_rows(rows(2, 1024, E, F32, std=0.1))
    status = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def step():
        n = pa.hstu_rmsnorm_fwd(x, eps=EPS, quant=True)
        return pa.hstu_uvqk_fp8_fwd(n["q8"], n["scale"], w8, ws, H, 128, 128, act=1,
                                    workspace=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (5, 6):
        x.copy_(rows(seed, T, E, BF16))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        for n in "uvqk":
            assert torch.equal(out[n], want[n])
    assert pa.hstu_attn_check(status) == 0
