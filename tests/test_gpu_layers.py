"""Layer norm, linear and their gradients against the fp64 oracle, on the GPU.

Tolerances, element by element, from the arithmetic (u = 2^-24, half a step of fp32):
  output rounding   half a step of the output's dtype, relative: 2^-8 bf16, 2^-24 fp32
  layer norm        sums of D values are formed in at most n = D / 256 + 40 additions per
                    value, so a mean is off by n u avg|x| and the other terms follow
  products          the tensor cores add 16 products at a time and truncate: one step,
                    2^-23, of the running sum each time, so K / 16 + 16 of them against
                    S = sum |a b|.  fp32 operands go in as three exact terms; the products
                    left out are below 2^-22 of S
  activations       2^-20 + z^2 2^-21 relative (exp, reciprocal and erfc to a few units, and
                    the rounding of their arguments, which weighs up to z^2)
  slopes            2^-19 (1 + |slope|)"""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import layers_oracle as lo
from tests.gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
FILL = 777.0  # what the bytes around a strided output hold


def f64(t):
    return t.detach().cpu().double().numpy()


def draw(gen, rows, cols, dtype, std=1.0, shift=0.0, pad=0):
    """rows x cols with rows of cols + pad elements."""
    t = torch.randn(rows, cols + pad, generator=gen) * std + shift
    return t.to(dtype).cuda()[:, :cols]


def framed(rows, cols, dtype, pad):
    """An output with `pad` more columns, 3 more rows behind, all FILL; and its frame."""
    buf = torch.full((rows + 3, cols + pad), FILL, dtype=dtype, device="cuda")
    return buf[:rows, :cols], buf


def frame_untouched(buf, rows, cols):
    assert (buf[rows:] == FILL).all() and (buf[:rows, cols:] == FILL).all()


def close(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / (tol + 1e-300), 0)), bad.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst at {i}: {got[i]!r} for {want[i]!r}, "
                             f"tolerance {np.broadcast_to(tol, bad.shape)[i]:.3e}")


# ------------------------------------------------------------------ layer norm

NORM_SIZES = [(1, 1), (1, 7), (2, 8), (3, 64), (5, 255), (1, 768), (130, 768), (67, 1000), (9, 1024), (4, 1025),
              (3, 4096), (2, 5000), (2, 8192), (2, 16400), (1, 40000)]


def norm_terms(D):
    return D / 256 + 40


def norm_tol(x, y, mean, rstd, gain, half):
    """|error| of y, mean, rstd."""
    n = norm_terms(x.shape[1])
    mx = np.abs(x).mean(1)
    e_mean = (n + 2) * U * mx
    d = x - mean[:, None]
    e_d = e_mean[:, None] + U * np.abs(d)
    # var: each square is off by 2 |d| e_d + u d^2, their sum by n u of itself; the mean of
    # d e_mean terms is second order, kept at first order as a bound
    var = (d * d).mean(1)
    e_var = (2 * np.abs(d) * e_d).mean(1) + (n + 4) * U * var
    e_r = rstd * (0.5 * e_var * rstd ** 2 + 4 * U)
    g = np.abs(gain)
    h = np.abs(d) * rstd[:, None]
    e_y = g * (e_d * rstd[:, None] + np.abs(d) * e_r[:, None] + 4 * U * h) + 4 * U * np.abs(y) + half * np.abs(y)
    return e_y + 1e-38, e_mean + 1e-38, e_r


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_layer_norm(rows, cols, dtype):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows * 1000 + cols)
    dt = DT[dtype]
    for pad, pdt, shift in ((0, torch.float32, 0.0), (8, torch.bfloat16, 3.0), (3, torch.float32, -0.5)):
        x = draw(gen, rows, cols, dt, 1.0, shift, pad)
        gain, bias = draw(gen, 1, cols, pdt, 0.3, 1.0)[0], draw(gen, 1, cols, torch.float32, 0.5)[0]
        y, buf = framed(rows, cols, dt, pad)
        got = api.layer_norm(x, gain, bias, out=y)
        assert got[0] is y
        ry, rm, rr = lo.layer_norm(f64(x), f64(gain), f64(bias))
        ty, tm, tr = norm_tol(f64(x), ry, rm, rr, f64(gain), HALF[dt])
        ty = ty + 4 * U * np.abs(f64(bias))
        close(y, ry, ty, "y")
        close(got[1], rm, tm, "mean")
        close(got[2], rr, tr, "rstd")
        frame_untouched(buf, rows, cols)


def test_layer_norm_without_gain_and_bias_and_far_from_zero():
    """A mean of 1000 standard deviations: E[x^2] - mean^2 would lose the variance."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(5)
    x = draw(gen, 16, 1500, torch.float32, 1.0, 1000.0)
    y, mean, rstd = api.layer_norm(x)
    ry, rm, rr = lo.layer_norm(f64(x))
    ty, tm, tr = norm_tol(f64(x), ry, rm, rr, np.ones(1500), U)
    close(y, ry, ty, "y")
    close(rstd, rr, tr, "rstd")
    assert np.abs(f64(y) - ry).max() < 1e-2
    c = torch.full((3, 768), 2.5, device="cuda")  # no variance: y = bias, rstd = eps^-1/2
    y, mean, rstd = api.layer_norm(c, None, None, eps=1e-6)
    assert (y == 0).all() and (mean == 2.5).all()
    assert np.allclose(f64(rstd), 1e3, rtol=1e-6)


def test_layer_norm_nonfinite_rows_stay_alone():
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(6)
    for dt in (torch.bfloat16, torch.float32):
        for D in (768, 1001, 5000):
            x = draw(gen, 6, D, dt)
            clean = api.layer_norm(x)[0].clone()
            x[1, 3], x[4, D - 1] = float("nan"), float("inf")
            y, mean, rstd = api.layer_norm(x)
            for r in range(6):
                if r in (1, 4):
                    assert torch.isnan(y[r]).all() and not torch.isfinite(mean[r])
                else:
                    assert torch.equal(y[r], clean[r])
            dx, dg, db = api.layer_norm_backward(torch.ones_like(x), x, mean, rstd)
            assert torch.isfinite(dx[[0, 2, 3, 5]]).all() and not torch.isfinite(dx[[1, 4]]).any()


def norm_grad_reference(dy, x, mean, rstd, gain, skip, half):
    """Oracle gradients and their tolerances."""
    D = x.shape[1]
    dx, dg, db = lo.layer_norm_backward(dy, x, mean, rstd, gain, skip)
    r = rstd[:, None]
    h = (x - mean[:, None]) * r
    e_h = 3 * U * (np.abs(x) + np.abs(mean[:, None])) * r
    q = np.abs(dy * gain)
    n = norm_terms(D) + 4
    aq, aqh = q.mean(1, keepdims=True), (q * np.abs(h)).mean(1, keepdims=True)
    e_aqh = n * U * aqh + (q * e_h).mean(1, keepdims=True)
    e = r * (6 * U * (q + aq + np.abs(h) * aqh) + n * U * aq + np.abs(h) * e_aqh + e_h * aqh)
    t_dx = e + half * np.abs(dx) + U * (np.abs(dx) + (0 if skip is None else np.abs(skip)))
    m = x.shape[0] / 2 + 40  # a column's sum is formed in at most this many additions per value
    t_dg = m * U * np.abs(dy * h).sum(0) + (np.abs(dy) * e_h).sum(0)
    t_db = m * U * np.abs(dy).sum(0)
    return dx, dg, db, t_dx + 1e-38, t_dg + 1e-38, t_db + 1e-38


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(0, 64), (700, 96), (2500, 40), (301, 2048)])
def test_layer_norm_backward(rows, cols, dtype):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows * 1000 + cols + 1)
    dt = DT[dtype]
    for pad, pdt, sdt, acc in ((0, torch.float32, None, False), (8, torch.bfloat16, dt, True),
                               (5, torch.float32, torch.float32, False)):
        x, dy = draw(gen, rows, cols, dt, 1.0, 0.5, pad), draw(gen, rows, cols, dt, 0.1, 0.01, pad)
        gain = draw(gen, 1, cols, pdt, 0.3, 1.0)[0]
        skip = None if sdt is None else draw(gen, rows, cols, sdt, 0.1, 0.0, pad)
        _, rm, rr = lo.layer_norm(f64(x)) if rows else (None, np.zeros(0), np.zeros(0))
        mean, rstd = torch.from_numpy(rm).float().cuda(), torch.from_numpy(rr).float().cuda()
        dg0, db0 = draw(gen, 1, cols, torch.float32)[0], draw(gen, 1, cols, torch.float32)[0]
        dg, db = dg0.clone(), db0.clone()
        dx, buf = framed(rows, cols, dt, pad)
        out = api.layer_norm_backward(dy, x, mean, rstd, gain, skip=skip, dx=dx, dgain=dg, dbias=db, accumulate=acc)
        assert out[0] is dx and out[1] is dg and out[2] is db
        frame_untouched(buf, rows, cols)
        if rows == 0:
            for got, old in ((dg, dg0), (db, db0)):
                assert torch.equal(got, old if acc else torch.zeros_like(old))
            continue
        rdx, rdg, rdb, tx, tg, tb = norm_grad_reference(f64(dy), f64(x), f64(mean), f64(rstd), f64(gain),
                                                        None if skip is None else f64(skip), HALF[dt])
        close(dx, rdx, tx, "dx")
        if acc:
            rdg, rdb = rdg + f64(dg0), rdb + f64(db0)
        close(dg, rdg, tg + 2 * U * (np.abs(rdg) + np.abs(f64(dg0))), "dgain")
        close(db, rdb, tb + 2 * U * (np.abs(rdb) + np.abs(f64(db0))), "dbias")


def test_layer_norm_backward_into_the_skip_gradient():
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(9)
    for dt, D in ((torch.bfloat16, 768), (torch.float32, 1023)):
        x, dy, skip = (draw(gen, 50, D, dt) for _ in range(3))
        _, mean, rstd = api.layer_norm(x)
        want = api.layer_norm_backward(dy, x, mean, rstd, skip=skip)
        got = api.layer_norm_backward(dy, x, mean, rstd, skip=skip, dx=skip)
        assert got[0] is skip
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ linear

# tokens, in, out: one token to several tiles of every kind, odd sizes, sides below a tile
LINEAR_SIZES = [(1, 1, 1), (1, 16, 40), (1, 1024, 512), (3, 50, 33), (16, 768, 96), (17, 256, 129), (33, 65, 700),
                (64, 512, 64), (100, 130, 258), (130, 64, 1000), (257, 770, 257), (300, 1030, 96), (512, 256, 512),
                (1000, 120, 72)]



def product_tol(a, b, k):
    """a [m, k], b [n, k]: tolerance of a b^T."""
    return (k / 16 + 16) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + 1e-38


def act_error(z, name):
    if name in ("none", "relu"):
        return np.zeros_like(z)
    return (2.0 ** -20 + np.minimum(z * z, 2.0 ** 10) * 2.0 ** -21) * np.abs(lo.act(z, name)) + 1e-36


def lipschitz(z, name):
    return {"none": 1.0, "relu": 1.0, "gelu": 1.13, "gelu_tanh": 1.13, "silu": 1.1}.get(name) or 2 * np.abs(z) + 1e-3


MIX = [("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f32", "f32", "f32"), ("bf16", "bf16", "f32"),
       ("f32", "bf16", "f32")]


@pytest.mark.parametrize("xt,wt,yt", MIX)
@pytest.mark.parametrize("rows,n_in,n_out", LINEAR_SIZES)
def test_linear(rows, n_in, n_out, xt, wt, yt):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows * 7 + n_in * 3 + n_out)
    k = (rows + n_in + n_out) % len(lo.ACTS)
    for pad, act, with_bias, rt, keep in ((0, lo.ACTS[k], True, None, False), (8, lo.ACTS[k - 1], False, yt, True),
                                          (3, lo.ACTS[k - 2], True, "f32", False)):
        x, w = draw(gen, rows, n_in, DT[xt], 1.0, 0.0, pad), draw(gen, n_out, n_in, DT[wt], n_in ** -0.5, 0.0, pad)
        bias = draw(gen, 1, n_out, DT[wt], 0.5)[0] if with_bias else None
        res = None if rt is None else draw(gen, rows, n_out, DT[rt], 1.0, 0.0, pad)
        y, buf = framed(rows, n_out, DT[yt], pad)
        z, zbuf = framed(rows, n_out, DT[yt], pad) if keep else (None, None)
        got = api.linear(x, w, bias, act=act, residual=res, out=y, preact=z)
        assert (got[0] is y and got[1] is z) if keep else got is y
        X, W = f64(x), f64(w)
        ry, rz = lo.linear(X, W, None if bias is None else f64(bias), act, None if res is None else f64(res))
        e_z = product_tol(X, W, n_in) + 2 * U * np.abs(rz) + (0 if bias is None else 2 * U * np.abs(f64(bias)))
        half = HALF[DT[yt]]
        e_y = (lipschitz(rz, act) * e_z + act_error(rz, act) + e_z * e_z * (act == "relu2")
               + 2 * U * (np.abs(ry) + (0 if res is None else np.abs(f64(res)))) + half * np.abs(ry))
        close(y, ry, e_y, f"y {act}")
        frame_untouched(buf, rows, n_out)
        if keep:
            close(z, rz, e_z + half * np.abs(rz), "z")
            frame_untouched(zbuf, rows, n_out)


@pytest.mark.parametrize("xt,wt,yt", MIX)
@pytest.mark.parametrize("rows,n_in,n_out", LINEAR_SIZES + [(2100, 70, 40), (0, 64, 96)])
def test_linear_backward(rows, n_in, n_out, xt, wt, yt):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows * 5 + n_in * 3 + n_out)
    k = (rows + n_in + n_out) % len(lo.ACTS)
    for pad, act, st, acc in ((0, lo.ACTS[k], None, False), (8, lo.ACTS[k - 1], yt, True), (3, "none", "f32", False)):
        dy, w = draw(gen, rows, n_out, DT[xt], 0.1, 0.0, pad), draw(gen, n_out, n_in, DT[wt], 0.2, 0.0, pad)
        z = draw(gen, rows, n_in, DT[xt], 1.0, 0.0, pad)
        x = torch.from_numpy(lo.act(f64(z), act)).to(DT[xt]).cuda()
        skip = None if st is None else draw(gen, rows, n_in, DT[st], 0.1, 0.0, pad)
        dx, xbuf = framed(rows, n_in, DT[yt], pad)
        dw0 = draw(gen, n_out, n_in, torch.float32)
        dw, wbuf = framed(n_out, n_in, torch.float32, pad)
        dw.copy_(dw0)
        db0 = draw(gen, 1, n_out, torch.float32)[0]
        db = db0.clone()
        got = api.linear_backward(dy, x, w, in_act=act, in_preact=z, skip=skip, dx=dx, dw=dw, db=db, accumulate=acc)
        assert got[0] is dx and got[1] is dw and got[2] is db
        for b, r, c in ((xbuf, rows, n_in), (wbuf, n_out, n_in)):
            frame_untouched(b, r, c)
        if rows == 0:
            assert torch.equal(dw, dw0 if acc else torch.zeros_like(dw0))
            assert torch.equal(db, db0 if acc else torch.zeros_like(db0))
            continue
        G, W, X, Z = f64(dy), f64(w), f64(x), f64(z)
        rdx, rdw, rdb = lo.linear_backward(G, X, W, act, Z, None if skip is None else f64(skip))
        slope = lo.act_slope(Z, act)
        plain = np.abs(G @ W)
        e = (product_tol(G, W.T, n_out) * np.abs(slope) + plain * (act not in ("none", "relu")) * 2.0 ** -19
             * (1 + np.abs(slope)))
        e = e + 2 * U * (np.abs(rdx) + (0 if skip is None else np.abs(f64(skip)))) + HALF[DT[yt]] * np.abs(rdx)
        close(dx, rdx, e + 1e-38, f"dx {act}")
        e_w = product_tol(G.T, X.T, rows)
        e_b = (rows / 2 + 40) * U * np.abs(G).sum(0) + 1e-38
        if acc:
            rdw, rdb = rdw + f64(dw0), rdb + f64(db0)
        close(dw, rdw, e_w + 2 * U * (np.abs(rdw) + np.abs(f64(dw0))), "dw")
        close(db, rdb, e_b + 2 * U * (np.abs(rdb) + np.abs(f64(db0))), "db")


# Sizes that the plan runs as CTA pairs, with and without a split reduction, and as small
# products together and apart; the odd ones leave output rows off 16 bytes.
LARGE_SIZES = [(256, 256, 8192), (4096, 256, 512), (2304, 768, 768), (1500, 2048, 2560), (1501, 2049, 1283),
               (40, 4096, 6000), (9000, 256, 264), (128, 5000, 128), (3, 3123, 4422)]


def tol64(a, b, k):
    return (k / 16 + 16) * 2.0 ** -23 * (a.abs() @ b.abs().t()) + 1e-38


def close64(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert got.shape == want.shape and not torch.isnan(off).any(), what
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.numel()} off, by up to {float(off.max()):.3e}"


@pytest.mark.parametrize("xt,wt,yt,act", [("bf16", "bf16", "bf16", "gelu"), ("bf16", "bf16", "f32", "silu"),
                                          ("f32", "f32", "f32", "relu2"), ("bf16", "f32", "bf16", "gelu_tanh")])
@pytest.mark.parametrize("rows,n_in,n_out", LARGE_SIZES)
def test_linear_large(rows, n_in, n_out, xt, wt, yt, act):
    """As test_linear and test_linear_backward, with the fp64 products taken on the GPU."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator(device="cuda").manual_seed(rows + n_in + n_out)

    def mk(r, c, dt, std):
        return (torch.randn(r, c, generator=gen, device="cuda") * std).to(DT[dt])

    on = lambda f, t, *a: torch.from_numpy(f(f64(t), *a)).cuda()  # noqa: E731
    half = HALF[DT[yt]]
    x, w, bias, res = mk(rows, n_in, xt, 1.0), mk(n_out, n_in, wt, n_in ** -0.5), mk(1, n_out, wt, 0.5)[0], mk(
        rows, n_out, yt, 1.0)
    y, z = torch.empty(rows, n_out, device="cuda", dtype=DT[yt]), torch.empty(rows, n_out, device="cuda", dtype=DT[yt])
    api.linear(x, w, bias, act=act, residual=res, out=y, preact=z)
    rz = x.double() @ w.double().t() + bias.double()
    e_z = tol64(x.double(), w.double(), n_in) + 2 * U * (rz.abs() + bias.double().abs())
    close64(z, rz, e_z + half * rz.abs(), "z")
    ry = on(lo.act, rz, act) + res.double()
    lip = 2 * rz.abs() + 1e-3 if act == "relu2" else 1.13
    e_y = lip * e_z + e_z * e_z + torch.from_numpy(act_error(f64(rz), act)).cuda()
    close64(y, ry, e_y + 2 * U * (ry.abs() + res.double().abs()) + half * ry.abs(), "y")

    dy, zin, skip = mk(rows, n_out, xt, 0.1), mk(rows, n_in, xt, 1.0), mk(rows, n_in, yt, 0.1)
    dw0 = torch.randn(n_out, n_in, generator=gen, device="cuda")
    db0 = torch.randn(n_out, generator=gen, device="cuda")
    dw, db, dx = dw0.clone(), db0.clone(), torch.empty(rows, n_in, device="cuda", dtype=DT[yt])
    api.linear_backward(dy, x, w, in_act=act, in_preact=zin, skip=skip, dx=dx, dw=dw, db=db, accumulate=True)
    g = dy.double()
    plain = g @ w.double()
    slope = on(lo.act_slope, zin, act)
    rdx = plain * slope + skip.double()
    e_x = tol64(g, w.double().t(), n_out) * slope.abs() + plain.abs() * 2.0 ** -19 * (1 + slope.abs())
    close64(dx, rdx, e_x + 2 * U * (rdx.abs() + skip.double().abs()) + half * rdx.abs() + 1e-38, "dx")
    rdw = g.t() @ x.double() + dw0.double()
    close64(dw, rdw, tol64(g.t(), x.double().t(), rows) + 2 * U * (rdw.abs() + dw0.double().abs()), "dw")
    rdb = g.sum(0) + db0.double()
    close64(db, rdb, (rows / 2 + 40) * U * g.abs().sum(0) + 2 * U * (rdb.abs() + db0.double().abs()), "db")
    # each gradient by itself is the same
    only = api.linear_backward(dy, x, w, need_dx=False, need_dw=False)[2]
    close64(only, g.sum(0), (rows / 2 + 40) * U * g.abs().sum(0) + 1e-38, "db alone")
    only = api.linear_backward(dy, x, w, need_dx=False, need_db=False)[1]
    close64(only, g.t() @ x.double(), tol64(g.t(), x.double().t(), rows), "dw alone")


@pytest.mark.parametrize("rows,n_in,n_out", [(200, 64, 200), (300, 4096, 136), (4096, 264, 136), (5, 2048, 64)])
def test_fp32_products_hold_fp32(rows, n_in, n_out):
    """fp32 operands and fp32 results: the Frobenius error stays at a few fp32 steps.

    The running sum is truncated once per 16 products, by at most 2^-23 of itself, in pieces
    of at most 1024 products that are then added with rounding; for zero-mean data a partial
    sum is on average no larger than the result.  So 64 truncations and 8 more steps for the
    terms left out and the joins: 72 * 2^-23.  A lost third term alone would be about 2^-17."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(11)
    x, w, dy = (draw(gen, *s, torch.float32) for s in ((rows, n_in), (n_out, n_in), (rows, n_out)))
    y = api.linear(x, w)
    dx, dw, _ = api.linear_backward(dy, x, w)
    ry, _ = lo.linear(f64(x), f64(w))
    rdx, rdw, _ = lo.linear_backward(f64(dy), f64(x), f64(w))
    for got, want, k in ((y, ry, n_in), (dx, rdx, n_out), (dw, rdw, rows)):
        steps = min(k / 16, 64) + 8
        assert np.linalg.norm(f64(got) - want) <= steps * 2.0 ** -23 * np.linalg.norm(want)


def test_bf16_products_into_fp32_gradients_hold_fp32():
    """dW from bf16 operands is an fp32 sum: long reductions do not drift (as above)."""
    require_gpu()
    from newton_schulz_11_b200 import api

    for rows, n_in, n_out, shift in ((12000, 128, 96, 0.0), (9000, 300, 272, 0.5)):
        gen = torch.Generator().manual_seed(rows)
        x, dy = (draw(gen, rows, c, torch.bfloat16, 1.0, shift) for c in (n_in, n_out))
        w = draw(gen, n_out, n_in, torch.bfloat16)
        _, dw, db = api.linear_backward(dy, x, w, need_dx=False)
        rdw = f64(dy).T @ f64(x)
        assert np.linalg.norm(f64(dw) - rdw) <= 72 * 2.0 ** -23 * np.linalg.norm(rdw)
        assert np.linalg.norm(f64(db) - f64(dy).sum(0)) <= 1e-5 * np.linalg.norm(f64(dy).sum(0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(0, 5), (1, 1), (1, 8), (3, 257), (64, 1000), (5, 4096), (33, 24)])
@pytest.mark.parametrize("act", lo.ACTS[1:])
def test_activation_backward(rows, cols, act, dtype):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows + cols)
    for pad, zt in ((0, dtype), (8, "bf16"), (3, "f32")):
        dy, z = draw(gen, rows, cols, DT[dtype], 1.0, 0.0, pad), draw(gen, rows, cols, DT[zt], 4.0, 0.0, pad)
        dz, buf = framed(rows, cols, DT[dtype], pad)
        assert api.activation_backward(dy, z, act, out=dz) is dz
        slope = lo.act_slope(f64(z), act)
        want = f64(dy) * slope
        tol = np.abs(f64(dy)) * 2.0 ** -19 * (1 + np.abs(slope)) + HALF[DT[dtype]] * np.abs(want)
        close(dz, want, tol + 1e-38, act)
        frame_untouched(buf, rows, cols)


def test_activation_slopes_at_the_ends():
    require_gpu()
    from newton_schulz_11_b200 import api

    inf = float("inf")
    z = torch.tensor([[0.0, -0.0, 1e30, -1e30, inf, -inf, 100.0, -100.0]], device="cuda")
    one = torch.ones_like(z)
    for act in ("gelu", "gelu_tanh", "silu"):
        d = api.activation_backward(one, z, act)[0].tolist()
        assert d == [0.5, 0.5, 1, 0, 1, 0, 1, 0], (act, d)
    assert api.activation_backward(one, z, "relu")[0].tolist() == [0, 0, 1, 0, 1, 0, 1, 0]
    nan = torch.full((1, 8), float("nan"), device="cuda")
    for act in lo.ACTS[2:]:
        assert torch.isnan(api.activation_backward(one, nan, act)).all(), act


def test_products_keep_nonfinite_rows_apart():
    """A NaN or an infinity in one token reaches that token's outputs only, and no bytes
    outside the operands (here NaN) reach any."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(3)
    for dt in (torch.bfloat16, torch.float32):
        for rows, n_in, n_out in ((5, 200, 72), (300, 200, 264)):
            frame = torch.full((rows + 8, n_in + 8), float("nan"), dtype=dt, device="cuda")
            x = frame[:rows, :n_in]
            x.copy_(draw(gen, rows, n_in, dt))
            wf = torch.full((n_out + 8, n_in + 8), float("nan"), dtype=dt, device="cuda")
            w = wf[:n_out, :n_in]
            w.copy_(draw(gen, n_out, n_in, dt))
            clean = api.linear(x, w)
            assert torch.isfinite(clean).all()
            dx, dw, db = api.linear_backward(clean, x, w)
            assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
            x[2, 5] = float("nan")
            x[4, 7] = float("inf")
            y = api.linear(x, w)
            keep = [r for r in range(rows) if r not in (2, 4)]
            assert torch.equal(y[keep], clean[keep])
            assert torch.isnan(y[2]).all() and not torch.isfinite(y[4]).any()


def test_large_fp32_values_survive():
    """The top of fp32's range does not overflow on its way into bf16 terms."""
    require_gpu()
    from newton_schulz_11_b200 import api

    x = torch.full((2, 16), 3.4e38, device="cuda")
    w = torch.zeros(3, 16, device="cuda")
    w[:, 3] = 0.5
    assert np.allclose(f64(api.linear(x, w)), 1.7e38, rtol=1e-6)


# ------------------------------------------------------------------ how they are called

def mlp_step(api, p, x, dout):
    """A pre-norm MLP sublayer, forward and backward, and its optimizer steps."""
    n, mean, rstd = api.layer_norm(x, p["gain"], p["beta"])
    h, z = api.linear(n, p["w1"], p["b1"], act="gelu_tanh", save_preact=True)
    y = api.linear(h, p["w2"], p["b2"], residual=x)
    dz, _, _ = api.linear_backward(dout, h, p["w2"], in_act="gelu_tanh", in_preact=z, dw=p["g_w2"], db=p["g_b2"])
    dn, _, _ = api.linear_backward(dz, n, p["w1"], dw=p["g_w1"], db=p["g_b1"])
    dx, _, _ = api.layer_norm_backward(dn, x, mean, rstd, p["gain"], skip=dout, dgain=p["g_gain"], dbias=p["g_beta"])
    return y, dx


def mlp_params(dt, d=256, hidden=512, seed=0):
    gen = torch.Generator().manual_seed(seed)
    p = {"gain": draw(gen, 1, d, torch.float32, 0.1, 1.0)[0], "beta": draw(gen, 1, d, torch.float32, 0.1)[0],
         "w1": draw(gen, hidden, d, dt, 0.05), "b1": draw(gen, 1, hidden, torch.float32, 0.1)[0],
         "w2": draw(gen, d, hidden, dt, 0.05), "b2": draw(gen, 1, d, torch.float32, 0.1)[0]}
    for k, s in (("w1", (hidden, d)), ("w2", (d, hidden)), ("b1", hidden), ("b2", d), ("gain", d), ("beta", d)):
        p["g_" + k] = torch.zeros(s, device="cuda")
    return p


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mlp_block_and_its_steps(dtype):
    """The operators in the order a training step uses them, against the oracle run on the
    same chain; then Muon and AdamW step the parameters from the gradients in place."""
    require_gpu()
    import oracle
    from newton_schulz_11_b200 import api
    from oracle import adamw_oracle as ao

    dt = DT[dtype]
    p = mlp_params(dt)
    gen = torch.Generator().manual_seed(1)
    x, dout = draw(gen, 200, 256, dt), draw(gen, 200, 256, dt, 0.1)
    y, dx = mlp_step(api, p, x, dout)
    P = {k: f64(v) for k, v in p.items()}
    n, mean, rstd = lo.layer_norm(f64(x), P["gain"], P["beta"])
    h, z = lo.linear(n, P["w1"], P["b1"], "gelu_tanh")
    ry, _ = lo.linear(h, P["w2"], P["b2"], "none", f64(x))
    dz, gw2, gb2 = lo.linear_backward(f64(dout), h, P["w2"], "gelu_tanh", z)
    dn, gw1, gb1 = lo.linear_backward(dz, n, P["w1"])
    rdx, gg, gbt = lo.layer_norm_backward(dn, f64(x), mean, rstd, P["gain"], f64(dout))
    # each tensor on the chain is rounded once, at most six in a row, each by half a step
    tol = 6 * HALF[dt] + 1e-6
    for got, want in ((y, ry), (dx, rdx), (p["g_w2"], gw2), (p["g_b2"], gb2), (p["g_w1"], gw1), (p["g_b1"], gb1),
                      (p["g_gain"], gg), (p["g_beta"], gbt)):
        assert np.linalg.norm(f64(got) - want) <= tol * np.linalg.norm(want)
    ws = [p["w1"], p["w2"]]
    moms = [torch.zeros_like(p["g_w1"]), torch.zeros_like(p["g_w2"])]
    old = [f64(w) for w in ws]
    api.muon_step(ws, [p["g_w1"], p["g_w2"]], moms, lr=0.02)
    for w, w0, k in zip(ws, old, ("g_w1", "g_w2")):
        want = oracle.muon_step(w0, f64(p[k]), np.zeros_like(w0), lr=0.02, beta=0.95, weight_decay=0.0,
                                nesterov=True, coeffs=[oracle.QUINTIC] * 5)[0]
        step = np.linalg.norm(want - w0)
        assert np.linalg.norm(f64(w) - want) <= 2e-2 * step + HALF[dt] * np.linalg.norm(want)
    vec = ["gain", "beta", "b1", "b2"]
    vs = [p[k] for k in vec]
    gs = [p["g_" + k] for k in vec]
    m, v = [torch.zeros_like(t) for t in vs], [torch.zeros_like(t) for t in vs]
    before = [f64(t) for t in vs]
    api.adamw_step(vs, gs, m, v, lr=1e-3, step=1)
    for t, b, g in zip(vs, before, gs):
        want = ao.adamw_step(b, f64(g), np.zeros_like(b), np.zeros_like(b), step=1, lr=1e-3, beta1=0.9, beta2=0.999,
                             eps=1e-8, weight_decay=0.0)[0]
        assert np.allclose(f64(t), want, rtol=1e-6, atol=1e-8)


def test_gradients_are_differences():
    """The GPU's own forward pass, differenced along one direction per tensor, in fp32."""
    require_gpu()
    from newton_schulz_11_b200 import api

    p = mlp_params(torch.float32, 96, 160)
    gen = torch.Generator().manual_seed(2)
    x, dout = draw(gen, 70, 96, torch.float32), draw(gen, 70, 96, torch.float32)
    _, dx = mlp_step(api, p, x, dout)
    grads = {k: f64(p["g_" + k]) for k in ("gain", "beta", "w1", "b1", "w2", "b2")}
    grads["x"] = f64(dx)

    def loss():
        n, _, _ = api.layer_norm(x, p["gain"], p["beta"])
        h = api.linear(n, p["w1"], p["b1"], act="gelu_tanh")
        return float((f64(api.linear(h, p["w2"], p["b2"], residual=x)) * f64(dout)).sum())

    for k, g in grads.items():
        t = x if k == "x" else p[k]
        v = torch.randn(t.shape, generator=gen)
        v = (v / v.norm()).cuda()
        keep, eps = t.clone(), 0.02 * float(t.norm() + 1)
        got = []
        for e in (eps, eps / 2):  # Richardson: the error falls to eps^4
            t.copy_(keep + e * v)
            a = loss()
            t.copy_(keep - e * v)
            got.append((a - loss()) / (2 * e))
            t.copy_(keep)
        d = (4 * got[1] - got[0]) / 3
        want = float((g * f64(v)).sum())
        scale = np.linalg.norm(g)
        # fp32 outputs: 6720 values of the loss, each off by a few 2^-24, over 2 eps
        assert abs(d - want) <= 2e-2 * scale + 1e-2 * abs(want), (k, d, want, scale)


def test_streams_and_explicit_buffers_agree():
    """Two streams at once, each with its own data, equal the same calls made one by one."""
    require_gpu()
    from newton_schulz_11_b200 import api

    def work(seed, stream=None):
        gen = torch.Generator().manual_seed(seed)
        x, w = draw(gen, 300, 515, torch.float32), draw(gen, 260, 515, torch.float32)
        g = draw(gen, 300, 260, torch.float32)
        torch.cuda.synchronize()
        out = []
        for _ in range(4):
            y = api.linear(x, w, act="silu", stream=stream)
            out = [y, *api.linear_backward(g, x, w, stream=stream), *api.layer_norm(x, stream=stream)]
            out += api.layer_norm_backward(x, x, out[5], out[6], stream=stream)
        return out

    want = [work(1), work(2)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [work(1, s[0]), work(2, s[1])]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_captured_and_replayed():
    """Two graphs captured apart (scratch of their own), replayed in turn and together on two
    streams, on new data in the same buffers."""
    require_gpu()
    from newton_schulz_11_b200 import api

    def one(seed, dt):
        p = mlp_params(dt, 264, 520, seed)
        gen = torch.Generator().manual_seed(seed)
        x, dout = draw(gen, 90, 264, dt), draw(gen, 90, 264, dt, 0.1)
        mlp_step(api, p, x, dout)  # outside the capture first
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, dx = mlp_step(api, p, x, dout)
        return p, x, dout, g, y, dx

    runs = [one(1, torch.float32), one(2, torch.bfloat16)]
    for p, x, dout, g, y, dx in runs:
        x.copy_(x.flip(0))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, r in zip(streams, runs):
            with torch.cuda.stream(s):
                r[3].replay()
    torch.cuda.synchronize()
    for p, x, dout, g, y, dx in runs:
        got = [y.clone(), dx.clone(), *(p[k].clone() for k in sorted(p) if k.startswith("g_"))]
        ey, edx = mlp_step(api, p, x, dout)
        for a, b in zip(got, [ey, edx, *(p[k] for k in sorted(p) if k.startswith("g_"))]):
            assert torch.equal(a, b)


def test_same_call_twice_gives_the_same_bits():
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(4)
    x, dy = draw(gen, 3000, 520, torch.bfloat16), draw(gen, 3000, 264, torch.bfloat16)
    w = draw(gen, 264, 520, torch.bfloat16)
    _, mean, rstd = api.layer_norm(x)

    def run():
        return [api.linear(x, w, act="gelu"), *api.linear_backward(dy, x, w),
                *api.layer_norm_backward(x, x, mean, rstd)]

    want = run()
    for _ in range(5):
        for a, b in zip(run(), want):
            assert torch.equal(a, b)


def test_only_what_is_asked_for():
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(8)
    x, dy, w = draw(gen, 40, 64, torch.bfloat16), draw(gen, 40, 96, torch.bfloat16), draw(gen, 96, 64, torch.bfloat16)
    dx, dw, db = api.linear_backward(dy, x, w)
    for k in range(3):
        need = [i == k for i in range(3)]
        got = api.linear_backward(dy, x, w, need_dx=need[0], need_dw=need[1], need_db=need[2])
        for i, want in enumerate((dx, dw, db)):
            assert got[i] is None if not need[i] else torch.equal(got[i], want)
    ws = api.Workspace(x.device)  # a caller's workspace serves every call, one after the other
    xf, wf, dyf = x.float(), w.float(), dy.float()
    want = [api.linear(xf, wf), *api.linear_backward(dyf, xf, wf)]
    got = [api.linear(xf, wf, workspace=ws), *api.linear_backward(dyf, xf, wf, workspace=ws)]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    r = draw(gen, 40, 96, torch.bfloat16)
    want = api.linear(x, w, residual=r)
    assert api.linear(x, w, residual=r, out=r) is r and torch.equal(r, want)
    s = draw(gen, 40, 64, torch.bfloat16)
    want = api.linear_backward(dy, x, w, skip=s)[0]
    assert api.linear_backward(dy, x, w, skip=s, dx=s)[0] is s and torch.equal(s, want)
    assert api.layers_status() == (0, 0)


def test_slices_of_one_buffer():
    """Column blocks of a fused buffer (as a packed QKV projection has) as inputs and outputs."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(12)
    big = torch.zeros(70, 3 * 128, dtype=torch.bfloat16, device="cuda")
    x, w = draw(gen, 70, 256, torch.bfloat16), [draw(gen, 128, 256, torch.bfloat16) for _ in range(3)]
    for i in range(3):
        api.linear(x, w[i], out=big[:, 128 * i:128 * (i + 1)])
    for i in range(3):
        assert torch.equal(big[:, 128 * i:128 * (i + 1)], api.linear(x, w[i]))
    y = api.linear(big[:, :128], draw(gen, 128, 128, torch.bfloat16), out=big[:, 128:256])
    assert y.shape == (70, 128)


def test_refusals_name_the_argument():
    require_gpu()
    from newton_schulz_11_b200 import api

    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    g = torch.zeros(4, 6, device="cuda")
    mean = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="w has shape"):
        api.linear(x, torch.zeros(6, 7, device="cuda"))
    with pytest.raises(ValueError, match="bias must be a contiguous vector"):
        api.linear(x, w, torch.zeros(5, device="cuda"))
    with pytest.raises(TypeError, match="x has dtype"):
        api.linear(x.half(), w)
    with pytest.raises(ValueError, match="unknown activation"):
        api.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="unit stride"):
        api.linear(torch.zeros(8, 4, device="cuda").t(), w)
    with pytest.raises(ValueError, match="must not repeat rows"):
        api.linear(torch.zeros(1, 8, device="cuda").expand(4, 8), w)
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        api.linear(x.cpu(), w)
    with pytest.raises(ValueError, match="residual is on"):
        api.linear(x, w, residual=g.cpu())
    with pytest.raises(api.MuonError):  # y may not lie over x
        api.linear(torch.zeros(4, 6, device="cuda"), torch.zeros(6, 6, device="cuda"), out=x.view(-1)[:24].view(4, 6),
                   residual=x.view(-1)[4:28].view(4, 6))
    with pytest.raises(ValueError, match="accumulate needs"):
        api.linear_backward(g, x, w, accumulate=True)
    with pytest.raises(ValueError, match="in_act needs in_preact"):
        api.linear_backward(g, x, w, in_act="gelu")
    with pytest.raises(TypeError, match="dw has dtype"):
        api.linear_backward(g, x, w, dw=torch.zeros(6, 8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="x must be 2-D"):
        api.layer_norm(torch.zeros(2, 3, 4, device="cuda"))
    with pytest.raises(TypeError, match="dy has dtype"):
        api.layer_norm_backward(x.bfloat16(), x, mean, mean)
    with pytest.raises(ValueError, match="mean must be"):
        api.layer_norm_backward(x, x, mean[:3], mean)
    with pytest.raises(api.MuonError):
        api.layer_norm(x, eps=float("nan"))
    with pytest.raises(api.MuonError):  # in place over the input is not offered
        api.layer_norm(x, out=x)


# sizes whose two products are small and share a launch: evenly, with different splits, with
# CTAs of the last cluster left over, and ragged
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,n_in,n_out", [(256, 640, 896), (130, 384, 640), (300, 520, 384), (512, 256, 1152),
                                             (1000, 136, 648), (129, 1160, 264), (777, 333, 259)])
def test_two_products_in_one_launch(rows, n_in, n_out, xt, wt):
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator(device="cuda").manual_seed(rows * n_out + n_in)

    def mk(r, c, dt, std):
        return (torch.randn(r, c, generator=gen, device="cuda") * std).to(DT[dt])

    dy, x, w = mk(rows, n_out, xt, 0.1), mk(rows, n_in, xt, 1.0), mk(n_out, n_in, wt, n_in ** -0.5)
    dx, dw, db = api.linear_backward(dy, x, w)
    g = dy.double()
    rdx, rdw, rdb = g @ w.double(), g.t() @ x.double(), g.sum(0)
    half = HALF[DT[xt]]
    close64(dx, rdx, tol64(g, w.double().t(), n_out) + (half + 2 * U) * rdx.abs() + 1e-38, "dx")
    close64(dw, rdw, tol64(g.t(), x.double().t(), rows) + 2 * U * rdw.abs(), "dw")
    close64(db, rdb, (rows / 2 + 40) * U * g.abs().sum(0) + 2 * U * rdb.abs(), "db")


def test_first_calls_of_a_process_are_captured():
    """Nothing has to run before the capture: the kernels load, the plans are made and the
    scratch is taken inside it."""
    require_gpu()
    code = """
import torch
from newton_schulz_11_b200 import api
torch.manual_seed(0)
x = torch.randn(200, 264, device="cuda")
w1, w2 = torch.randn(520, 264, device="cuda") / 16, torch.randn(264, 520, device="cuda").bfloat16() / 16
gain = torch.ones(264, device="cuda")
def step():
    n, mean, rstd = api.layer_norm(x, gain)
    h, z = api.linear(n, w1, act="gelu", save_preact=True)
    y = api.linear(h, w2, residual=x)
    dz, dw2, db2 = api.linear_backward(y, h, w2, in_act="gelu", in_preact=z)
    dn, dw1, db1 = api.linear_backward(dz, n, w1)
    a = api.activation_backward(dz, z, "silu")
    return [y, dw2, db2, dw1, db1, a, *api.layer_norm_backward(dn, x, mean, rstd, gain, skip=y)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = step()
for t in out:
    t.fill_(float("nan"))
g.replay()
x.copy_(x.flip(0))
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step()))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]
