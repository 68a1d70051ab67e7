"""Bounded waits of the layer kernels: a wait that runs out is reported by layers_status and
the context stays usable.  The failure is made by a wait budget far shorter than any copy
takes, never by a fault or a trap; the kernels wait for their own copies and MMAs, up to two
seconds, and leave.  The budget is looked at every 32 polls, and a poll sleeps until its
barrier or a time of the hardware's own: a wait that ends before that has not run out, so
the kernels with short waits may as well finish, correctly.  A large product's always do
run out."""
import pytest

from tests.gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["pair", "pair split", "small", "small cluster", "few tokens", "norm", "wide norm",
                                  "norm backward"])
def test_short_wait_budget_is_reported_and_recovered(what):
    require_gpu()
    from newton_schulz_11_b200 import _lib, api

    gen = torch.Generator(device="cuda").manual_seed(0)

    def mk(r, c, dtype=torch.bfloat16):
        return torch.randn(r, c, generator=gen, device="cuda").to(dtype)

    if what == "norm backward":
        x = mk(4000, 768)
        _, mean, rstd = api.layer_norm(x)
        run = lambda: api.layer_norm_backward(x, x, mean, rstd)  # noqa: E731
    elif "norm" in what:
        x = mk(4000, 768 if what == "norm" else 8192)
        run = lambda: api.layer_norm(x)  # noqa: E731
    else:
        rows, n_in, n_out = {"pair": (4096, 1024, 1024), "pair split": (512, 8192, 512), "small": (1024, 256, 1024),
                             "small cluster": (128, 1024, 256), "few tokens": (3, 4096, 1024)}[what]
        x, w = mk(rows, n_in), mk(n_out, n_in)
        run = lambda: (api.linear(x, w),)  # noqa: E731
    want = [t.clone() for t in run()]
    assert api.layers_status(clear=True) == (_lib.MUON_OK, 0)
    try:
        _lib.lib().muon_set_wait_timeout_us(1)
        got = run()
        code, where = api.layers_status()
        if code == _lib.MUON_OK:
            assert "pair" not in what
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        else:
            assert code == _lib.MUON_ERR_TIMEOUT and 1 <= where <= 5, (code, where)
        assert api.layers_status(clear=True) == (code, where)  # kept until cleared
    finally:
        _lib.lib().muon_set_wait_timeout_us(0)
    assert api.layers_status() == (_lib.MUON_OK, 0)
    for a, b in zip(run(), want):
        assert torch.equal(a, b)
    assert api.layers_status() == (_lib.MUON_OK, 0)
