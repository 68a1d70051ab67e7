"""Calls of the layers that once gave a wrong answer, on the GPU: each test fails on the code
that had the fault.

Tolerances as in test_gpu_layers.py, counted in u = 2^-24, half a step of fp32."""
import numpy as np
import pytest

from oracle import layers_oracle as lo
from tests.gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("cols", [2048, 2050])
def test_long_reductions_into_bf16_do_not_drift(cols):
    """The tensor cores truncate when they add 16 products to the accumulator; for products of one
    sign that is a drift, of less than two steps 2^-23 of the running sum each time.  In pieces
    of 2048 of k (128 additions), with a running sum that is half of the piece's on average, the
    result is too small by at most 128 * 2^-23 = 1.5e-5 relative; 2^17 of k in one piece lost
    7.8e-4.  The results' own rounding to bf16 is as often up as down (rows and columns are
    scaled so that the results spread over more than an octave): its mean over N results has a
    deviation of at most 2^-8 / sqrt(3 N), counted five times.  2048 columns take the plain
    tiles, 2050 the flipped ones."""
    require_gpu()
    from newton_schulz_11_b200 import api

    rows, k = 2304, 1 << 17
    gen = torch.Generator(device="cuda").manual_seed(17)

    def mk(n):
        t = torch.rand(n, k, generator=gen, device="cuda").add_(0.5)
        return t.mul_(torch.exp2(torch.rand(n, 1, generator=gen, device="cuda"))).bfloat16()

    x, w = mk(rows), mk(cols)
    got = {"y": api.linear(x, w), "dx": api.linear_backward(x, w.new_empty(rows, cols), w.t().contiguous(),
                                                            need_dw=False, need_db=False)[0]}
    want = torch.zeros(rows, cols, device="cuda", dtype=torch.float64)
    for i in range(0, k, 8192):
        want += x[:, i:i + 8192].double() @ w[:, i:i + 8192].double().t()
    for name, y in got.items():
        drift = float(((y.double() - want) / want).mean())
        assert abs(drift) <= 128 * 2.0 ** -23 + 5 * 2.0 ** -8 / (3 * want.numel()) ** 0.5, (name, drift)


def test_a_workspace_shared_with_the_step_keeps_its_status():
    """The step records a non-finite gradient in the workspace's first bytes, once, until they
    are cleared: layers that use the same workspace neither overwrite nor block that."""
    require_gpu()
    from newton_schulz_11_b200 import _lib, api

    gen = torch.Generator(device="cuda").manual_seed(1)

    def mk(r, c):
        return torch.randn(r, c, generator=gen, device="cuda")

    ws = api.Workspace(torch.device("cuda", torch.cuda.current_device()))
    ws.ensure(64 << 20, torch.cuda.current_stream().cuda_stream)
    p, g, m = mk(96, 64).bfloat16(), mk(96, 64), torch.zeros(96, 64, device="cuda")
    x, w, dy = mk(700, 520), mk(264, 520), mk(700, 264)
    _, mean, rstd = api.layer_norm(x)

    def layers(workspace):
        return [api.linear(x, w, workspace=workspace), *api.linear_backward(dy, x, w, workspace=workspace),
                *api.layer_norm_backward(x, x, mean, rstd, workspace=workspace)]

    want = layers(None)
    for a, b in zip(layers(ws), want):
        assert torch.equal(a, b)
    assert api.device_status(ws) == (_lib.MUON_OK, 0) and api.nonfinite_count(ws) == 0
    g[5, 7] = float("nan")
    api.muon_step([p], [g], [m], lr=0.02, workspace=ws)
    assert api.device_status(ws) == (_lib.MUON_ERR_NONFINITE, 0) and api.nonfinite_count(ws) == 1
    for a, b in zip(layers(ws), want):
        assert torch.equal(a, b)
    assert api.device_status(ws) == (_lib.MUON_ERR_NONFINITE, 0) and api.nonfinite_count(ws) == 1


def test_a_workspace_elsewhere_is_refused():
    """Before anything is queued, also by calls that need no scratch."""
    require_gpu()
    from newton_schulz_11_b200 import api

    x, w, dy = (torch.ones(s, device="cuda") for s in ((40, 64), (96, 64), (40, 96)))
    mean, rstd = torch.zeros(40, device="cuda"), torch.ones(40, device="cuda")
    here = torch.cuda.current_device()

    def calls(ws):
        yield lambda: api.linear(x, w, workspace=ws)
        yield lambda: api.linear(x.bfloat16(), w.bfloat16(), workspace=ws)
        yield lambda: api.linear_backward(dy, x, w, workspace=ws)
        yield lambda: api.layer_norm_backward(x, x, mean, rstd, workspace=ws)

    moved = api.Workspace("cuda")
    moved.buf = torch.empty(1 << 20, dtype=torch.uint8)  # its buffer says where it is
    for ws in (api.Workspace(f"cuda:{here + 1}"), api.Workspace("cpu"), moved):
        for call in calls(ws):
            with pytest.raises(ValueError, match="workspace is on"):
                call()
        assert ws is moved or ws.buf is None
    for call in calls("scratch"):
        with pytest.raises(TypeError, match="must be a Workspace"):
            call()
    for ws in (api.Workspace("cuda"), api.Workspace(f"cuda:{here}")):
        for _ in range(2):  # without and with a buffer
            for call in calls(ws):
                call()
        assert ws.buf.device == x.device


# (a bf16 row 1e4 standard deviations from zero has no two different values, and no rstd)
FAR = [(64, 768, 1000.0), (37, 1023, 1000.0), (3, 8192, 1000.0), (2, 16400, 1000.0), (50, 257, 0.0)]


@pytest.mark.parametrize("rows,cols,far,dtype", [(*c, d) for c in FAR for d in ("f32", "bf16")]
                         + [(40, 4096, 1e4, "f32")])
def test_norm_gradients_far_from_zero(rows, cols, far, dtype):
    """A mean of `far` standard deviations costs the gradients nothing: x - mean is formed first,
    where it rounds once, relative to itself.

    With u = 2^-24 and h = (x - mean) rstd: |error of h| <= 2 u |h|.  dgain: a column's sum takes
    at most rows + 8 additions.  dx = rstd (q - avg q - h avg(q h)): q, each average (in
    n = D / 256 + 44 additions at most) and the three operations that join them."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator().manual_seed(rows + cols)
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    half = {"f32": U, "bf16": 2.0 ** -8}[dtype]
    spread = 1.0 if dtype == "f32" else max(1.0, far / 16)
    x = (torch.randn(rows, cols, generator=gen) * spread + far * spread).to(dt).cuda()
    dy = (torch.randn(rows, cols, generator=gen) * 0.1).to(dt).cuda()
    gain = (torch.randn(cols, generator=gen) * 0.3 + 1).cuda()
    X, G, Q = f64(x), f64(gain), f64(dy) * f64(gain)
    mean = torch.from_numpy(X.mean(1)).float().cuda()
    rstd = torch.from_numpy(1 / X.std(1)).float().cuda()
    dx, dg, db = api.layer_norm_backward(dy, x, mean, rstd, gain)
    rdx, rdg, rdb = lo.layer_norm_backward(f64(dy), X, f64(mean), f64(rstd), G)
    r = f64(rstd)[:, None]
    h = np.abs(X - f64(mean)[:, None]) * r
    q = np.abs(Q)
    n = cols / 256 + 44
    aq, aqh = q.mean(1, keepdims=True), (q * h).mean(1, keepdims=True)
    t_dx = U * r * (6 * (q + aq + h * aqh) + n * aq + (n + 4) * h * aqh) + (half + U) * np.abs(rdx)
    assert (np.abs(f64(dx) - rdx) <= t_dx + 1e-38).all(), "dx"
    t_dg = (rows + 8 + 3) * U * (np.abs(f64(dy)) * h).sum(0)
    assert (np.abs(f64(dg) - rdg) <= t_dg + 1e-38).all(), "dgain"
    assert (np.abs(f64(db) - rdb) <= (rows + 8) * U * np.abs(f64(dy)).sum(0) + 1e-38).all(), "dbias"


MIXED = [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")]
# few tokens, small products (one CTA a tile, and clusters), pairs, pairs with a split
# reduction, and outputs whose rows are not 16-byte aligned
SIZES = [(3, 520, 264), (130, 200, 72), (300, 2000, 264), (2400, 512, 2304), (512, 8192, 512), (301, 203, 261),
         (2401, 515, 2305)]


@pytest.mark.parametrize("xt,wt", MIXED)
@pytest.mark.parametrize("rows,n_in,n_out", SIZES)
def test_infinities_meet_every_term(rows, n_in, n_out, xt, wt):
    """An infinite operand gives infinities and NaNs exactly where the sum in 64 bits has them:
    against values that are one bf16 term, values that are two or three, and zeros."""
    require_gpu()
    from newton_schulz_11_b200 import api

    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(rows + n_in)
    inf = float("inf")

    def mk(r, c, dtype):
        t = torch.randn(r, c, generator=gen, device="cuda")
        pick = torch.rand(r, c, generator=gen, device="cuda")
        t = torch.where(pick < 0.4, t.bfloat16().float(), t)               # one term
        t = torch.where(pick < 0.2, t.sign() * (1 + 2.0 ** -9), t)         # two
        t = torch.where(pick < 0.1, t.sign() * 2.0 ** -70, t)
        t = torch.where(pick < 0.05, torch.zeros_like(t), t)
        return t.to(dt[dtype])

    def same(got, want, what):
        got = got.double()
        assert torch.equal(torch.isnan(got), torch.isnan(want)), what
        assert torch.equal(got == inf, want == inf) and torch.equal(got == -inf, want == -inf), what

    x, w, dy = mk(rows, n_in, xt), mk(n_out, n_in, wt), mk(rows, n_out, xt)
    x[0, 5], x[rows // 2, n_in - 1], w[n_out // 3, 17] = inf, -inf, inf
    x[rows - 1, 3], x[rows - 1, 170] = inf, -inf
    out = torch.empty(rows, n_out, device="cuda")
    same(api.linear(x, w, out=out), x.double() @ w.double().t(), "y")
    same(api.linear(x, w), x.double() @ w.double().t(), "y in the dtype of x")
    dy[rows // 3, 2] = -inf
    dx, dw, db = api.linear_backward(dy, x, w)
    same(dx, dy.double() @ w.double(), "dx")
    same(dw, dy.double().t() @ x.double(), "dw")
    same(db, dy.double().sum(0), "db")


@pytest.mark.parametrize("xt,wt", MIXED)
@pytest.mark.parametrize("rows,n_in,n_out", SIZES)
def test_whole_numbers_stay_exact(rows, n_in, n_out, xt, wt):
    """Products of whole numbers below 2^8 (one bf16 term each) whose every partial sum is below
    2^24 have nothing to round or to truncate, and the terms that stand for nothing add 2^-59 to
    the sum, far below its half step."""
    require_gpu()
    from newton_schulz_11_b200 import api

    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, w, dy = (torch.randint(-31, 32, s, generator=gen, device="cuda").to(dt[t])
                for s, t in (((rows, n_in), xt), ((n_out, n_in), wt), ((rows, n_out), xt)))
    y, dx = torch.empty(rows, n_out, device="cuda"), torch.empty(rows, n_in, device="cuda")
    _, dw, db = api.linear_backward(dy, x, w, dx=dx)
    for got, want in ((api.linear(x, w, out=y), x.double() @ w.double().t()), (dx, dy.double() @ w.double()),
                      (dw, dy.double().t() @ x.double()), (db, dy.double().sum(0))):
        assert torch.equal(got.double(), want)


@pytest.mark.parametrize("rows,cols", [(50, 768), (20, 1023), (9, 9000), (0, 64)])
def test_norm_gradients_that_are_asked_for(rows, cols):
    """Each alone and in pairs, and a norm without a bias that accumulates its gain's gradient."""
    require_gpu()
    from newton_schulz_11_b200 import api

    gen = torch.Generator(device="cuda").manual_seed(cols)
    x, dy, skip = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(3))
    _, mean, rstd = api.layer_norm(x)
    names = ("need_dx", "need_dgain", "need_dbias")
    want = api.layer_norm_backward(dy, x, mean, rstd, skip=skip)
    for mask in range(1, 8):
        need = {n: bool(mask >> i & 1) for i, n in enumerate(names)}
        got = api.layer_norm_backward(dy, x, mean, rstd, skip=skip, **need)
        for i, n in enumerate(names):
            assert torch.equal(got[i], want[i]) if need[n] else got[i] is None
    for i, (kw, no) in enumerate(((dict(dgain=want[1].clone()), "need_dbias"), (dict(dbias=want[2].clone()), "need_dgain"))):
        got = api.layer_norm_backward(dy, x, mean, rstd, accumulate=True, **{no: False}, **kw)
        assert got[2 - i] is None and torch.equal(got[1 + i], want[1 + i] + want[1 + i])
        with pytest.raises(ValueError, match="accumulate needs"):
            api.layer_norm_backward(dy, x, mean, rstd, accumulate=True, **kw)
    with pytest.raises(ValueError, match="nothing to compute"):
        api.layer_norm_backward(dy, x, mean, rstd, **dict.fromkeys(names, False))
