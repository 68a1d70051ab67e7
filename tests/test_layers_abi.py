"""Layer entry points, host side (no GPU needed): argument checks with fake device pointers.
Nothing reaches a device; a valid call stops at the device check."""
import ctypes

import pytest

from newton_schulz_11_b200 import _lib
from newton_schulz_11_b200._lib import MUON_BF16, MUON_F32
from tests.conftest import cuda_present

E = _lib
BASE = 1 << 40
STEP = 1 << 34


@pytest.fixture(scope="module")
def L():
    from newton_schulz_11_b200 import build

    build.build()
    return _lib.lib()


def put(d, name, slot, ld, dtype=MUON_BF16):
    setattr(d, name + "_data", BASE + slot * STEP)
    setattr(d, name + "_ld", ld)
    setattr(d, name + "_dtype", dtype)


def norm(rows=4, cols=8):
    d = _lib.MuonLayerNorm(rows=rows, cols=cols, eps=1e-5)
    for i, n in enumerate(("x", "gain", "bias", "y")):
        put(d, n, i, cols)
    d.mean, d.rstd = BASE + 5 * STEP, BASE + 6 * STEP
    return d


def norm_grad(rows=4, cols=8):
    d = _lib.MuonLayerNormGrad(rows=rows, cols=cols)
    for i, n in enumerate(("dy", "x", "gain", "skip", "dx")):
        put(d, n, i, cols)
    for i, n in enumerate(("mean", "rstd", "dgain", "dbias")):
        setattr(d, n, BASE + (6 + i) * STEP)
    return d


def linear(rows=4, n_in=8, n_out=16):
    d = _lib.MuonLinear(rows=rows, in_features=n_in, out_features=n_out, act=_lib.MUON_ACTS["gelu"])
    for i, (n, ld) in enumerate((("x", n_in), ("w", n_in), ("bias", n_out), ("residual", n_out), ("y", n_out),
                                 ("preact", n_out))):
        put(d, n, i, ld)
    return d


def linear_grad(rows=4, n_in=8, n_out=16):
    d = _lib.MuonLinearGrad(rows=rows, in_features=n_in, out_features=n_out, in_act=_lib.MUON_ACTS["silu"])
    for i, (n, ld) in enumerate((("dy", n_out), ("x", n_in), ("w", n_in), ("preact", n_in), ("skip", n_in),
                                 ("dx", n_in), ("dw", n_in))):
        put(d, n, i, ld, MUON_F32 if n == "dw" else MUON_BF16)
    d.db = BASE + 8 * STEP
    return d


def act_grad(rows=4, cols=8):
    d = _lib.MuonActivationGrad(rows=rows, cols=cols, act=1)
    for i, n in enumerate(("dy", "z", "dz")):
        put(d, n, i, cols)
    return d


WS = BASE + 12 * STEP
MAKE = {"muon_layer_norm": norm, "muon_layer_norm_backward": norm_grad, "muon_linear": linear,
        "muon_linear_backward": linear_grad, "muon_activation_backward": act_grad}


def call(L, name, d, ws=WS, ws_bytes=1 << 32):
    f = getattr(L, name)
    return f(ctypes.byref(d), None) if len(f.argtypes) == 2 else f(ctypes.byref(d), ws, ws_bytes, None)


def refused(L, name, want, **fields):
    d = MAKE[name]()
    for k, v in fields.items():
        setattr(d, k, v)
    assert call(L, name, d) == want, (name, fields)


@pytest.mark.parametrize("name", MAKE)
def test_a_valid_call_reaches_the_device_check(L, name):
    if cuda_present():
        pytest.skip("fake device pointers: only where no kernel can run")
    for rows in (0, 1, 4, 5000):
        assert call(L, name, MAKE[name](rows)) in (E.MUON_ERR_NO_DEVICE, E.MUON_ERR_CUDA)


@pytest.mark.parametrize("name", MAKE)
def test_null_descriptor_and_sizes(L, name):
    f = getattr(L, name)
    assert (f(None, None) if len(f.argtypes) == 2 else f(None, None, 0, None)) == E.MUON_ERR_INVALID_ARG
    side = ["cols"] if "cols" in dict(MAKE[name]()._fields_) else ["in_features", "out_features"]
    for k in side:
        for v in (0, -1, (1 << 24) + 1):
            refused(L, name, E.MUON_ERR_UNSUPPORTED_SHAPE, **{k: v})
    for v in (-1, (1 << 30) + 1):
        refused(L, name, E.MUON_ERR_UNSUPPORTED_SHAPE, rows=v)


@pytest.mark.parametrize("name,views", [
    ("muon_layer_norm", ("x", "y")), ("muon_layer_norm_backward", ("dy", "x", "dx", "skip")),
    ("muon_linear", ("x", "w", "residual", "y", "preact")),
    ("muon_linear_backward", ("dy", "x", "w", "preact", "skip", "dx", "dw")),
    ("muon_activation_backward", ("dy", "z", "dz"))])
def test_views(L, name, views):
    for v in views:
        refused(L, name, E.MUON_ERR_UNSUPPORTED_SHAPE, **{v + "_ld": 7})
        refused(L, name, E.MUON_ERR_UNSUPPORTED_DTYPE, **{v + "_dtype": 2})
        refused(L, name, E.MUON_ERR_ALIGNMENT, **{v + "_data": BASE + 40 * STEP + 1})
        if v not in ("skip", "residual", "preact", "dx", "dw"):
            refused(L, name, E.MUON_ERR_INVALID_ARG, **{v + "_data": None})


def test_written_views_overlap_nothing(L):
    inv = E.MUON_ERR_INVALID_ARG
    refused(L, "muon_layer_norm", inv, y_data=BASE)
    refused(L, "muon_layer_norm", inv, y_data=BASE + 62)  # the last element of x
    refused(L, "muon_layer_norm", inv, rstd=BASE + 5 * STEP + 12)  # the last element of mean
    refused(L, "muon_layer_norm_backward", inv, dx_data=BASE)
    refused(L, "muon_layer_norm_backward", inv, dbias=BASE + 8 * STEP)
    refused(L, "muon_layer_norm_backward", inv, dx_data=WS)
    refused(L, "muon_linear", inv, y_data=BASE)
    refused(L, "muon_linear", inv, preact_data=BASE + 4 * STEP)
    refused(L, "muon_linear", inv, y_data=BASE + 3 * STEP + 2)  # beside the residual, not on it
    refused(L, "muon_linear_backward", inv, dx_data=BASE + 6 * STEP)
    refused(L, "muon_linear_backward", inv, db=BASE)
    refused(L, "muon_activation_backward", inv, dz_data=BASE)
    # the same rows with another dtype or stride are not the same view
    refused(L, "muon_linear", inv, y_data=BASE + 3 * STEP, y_dtype=MUON_F32)
    refused(L, "muon_linear", inv, y_data=BASE + 3 * STEP, y_ld=24)


def test_allowed_overlaps(L):
    if cuda_present():
        pytest.skip("fake device pointers: only where no kernel can run")
    ok = (E.MUON_ERR_NO_DEVICE, E.MUON_ERR_CUDA)
    d = linear()
    d.y_data = d.residual_data
    assert call(L, "muon_linear", d) in ok
    d = linear_grad()
    d.dx_data = d.skip_data
    assert call(L, "muon_linear_backward", d) in ok
    d = norm_grad()
    d.dx_data = d.skip_data
    assert call(L, "muon_layer_norm_backward", d) in ok
    d = linear()  # column blocks of one buffer, rows interleaved
    for n, off in (("x", 0), ("residual", 8), ("y", 24), ("preact", 40)):
        setattr(d, n + "_data", BASE + 2 * off)
        setattr(d, n + "_ld", 64)
    assert call(L, "muon_linear", d) in ok
    d.preact_data = BASE + 2 * 39
    assert call(L, "muon_linear", d) == E.MUON_ERR_INVALID_ARG
    d = linear_grad()  # inputs may overlap one another
    d.x_data = d.w_data = d.preact_data
    assert call(L, "muon_linear_backward", d) in ok


def test_options(L):
    for v in (-1, 6):
        refused(L, "muon_linear", E.MUON_ERR_INVALID_ARG, act=v)
        refused(L, "muon_linear_backward", E.MUON_ERR_INVALID_ARG, in_act=v)
        refused(L, "muon_activation_backward", E.MUON_ERR_INVALID_ARG, act=v)
    refused(L, "muon_activation_backward", E.MUON_ERR_INVALID_ARG, act=0)
    for v in (-1, 2):
        refused(L, "muon_linear_backward", E.MUON_ERR_INVALID_ARG, accumulate=v)
        refused(L, "muon_layer_norm_backward", E.MUON_ERR_INVALID_ARG, accumulate=v)
    for v in (float("nan"), float("inf"), -1e-5):
        refused(L, "muon_layer_norm", E.MUON_ERR_INVALID_ARG, eps=v)
    refused(L, "muon_layer_norm", E.MUON_ERR_UNSUPPORTED_DTYPE, y_dtype=MUON_F32)
    refused(L, "muon_layer_norm_backward", E.MUON_ERR_UNSUPPORTED_DTYPE, dx_dtype=MUON_F32)
    refused(L, "muon_linear_backward", E.MUON_ERR_UNSUPPORTED_DTYPE, dw_dtype=MUON_BF16)
    refused(L, "muon_activation_backward", E.MUON_ERR_UNSUPPORTED_DTYPE, dz_dtype=MUON_F32)
    refused(L, "muon_linear_backward", E.MUON_ERR_INVALID_ARG, preact_data=None)  # in_act needs it for dx
    refused(L, "muon_linear_backward", E.MUON_ERR_INVALID_ARG, dx_data=None, dw_data=None, db=None)
    refused(L, "muon_layer_norm_backward", E.MUON_ERR_INVALID_ARG, dx_data=None, dgain=None, dbias=None)


def test_workspace(L):
    d = norm_grad(5000, 512)
    n = ctypes.c_size_t(0)
    assert L.muon_layer_norm_backward_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert call(L, "muon_layer_norm_backward", d, WS, n.value - 1) == E.MUON_ERR_WORKSPACE_TOO_SMALL
    assert call(L, "muon_layer_norm_backward", d, None, n.value) == E.MUON_ERR_WORKSPACE_TOO_SMALL
    assert call(L, "muon_layer_norm_backward", d, WS + 4, n.value) == E.MUON_ERR_ALIGNMENT
    d.dgain = d.dbias = None
    assert L.muon_layer_norm_backward_workspace(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value == 0
    for name in ("muon_linear", "muon_linear_backward", "muon_layer_norm_backward"):
        assert getattr(L, name + "_workspace")(None, ctypes.byref(n)) == E.MUON_ERR_INVALID_ARG
        assert getattr(L, name + "_workspace")(ctypes.byref(MAKE[name]()), None) == E.MUON_ERR_INVALID_ARG
        assert getattr(L, name + "_workspace")(ctypes.byref(MAKE[name](rows=-1)), ctypes.byref(n)) \
            == E.MUON_ERR_UNSUPPORTED_SHAPE


def test_descriptor_sizes_match_the_header():
    assert ctypes.sizeof(_lib.MuonLayerNorm) == 136
    assert ctypes.sizeof(_lib.MuonLayerNormGrad) == 176
    assert ctypes.sizeof(_lib.MuonLinear) == 176
    assert ctypes.sizeof(_lib.MuonLinearGrad) == 208
    assert ctypes.sizeof(_lib.MuonActivationGrad) == 96


def test_python_refusals_without_a_gpu():
    torch = pytest.importorskip("torch")
    from newton_schulz_11_b200 import api

    x = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.linear(x, torch.zeros(3, 4))
    with pytest.raises(ValueError, match="2-D"):
        api.layer_norm(torch.zeros(4))
    with pytest.raises(TypeError, match="torch.Tensor"):
        api.layer_norm([1.0])
    with pytest.raises(ValueError, match="CUDA"):
        api.linear_backward(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        api.activation_backward(x, x, "gelu")
