"""How many bits fp32 results of long reductions hold, on the GPU.

The tensor cores truncate at each addition of 16 products, half a step 2^-23 of the running sum
on average.  For zero-mean products the running sum of a piece is on average 2/3 of the piece's
own size (the mean of sqrt t over 0..1), and pieces are independent, so the relative Frobenius
error of the whole is that of a piece:

  256 of k, an fp32 operand among the two    16 * 2/3 * 2^-24 = 6.4e-7
  512 of k, two bf16 operands                32 * 2/3 * 2^-24 = 1.28e-6

The n sums of the pieces are added with rounding to nearest, at most half a step 2^-24 each of
sums that grow like sqrt t: independent, sqrt(n / 2) 2^-24 at most.  A lost third term of an
operand is about 2^-17, and a reduction of 8192 in one piece about 9e-6."""
import pytest

from tests.gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu

# large products of one and two waves of pairs, one with a split reduction, and small ones with
# one CTA a tile and with clusters
SIZES = [(2400, 8192, 2304), (4096, 8192, 2304), (512, 16384, 512), (1500, 8192, 1500), (300, 16384, 136),
         (9, 8192, 600), (2401, 8193, 2305)]


@pytest.mark.parametrize("xt,wt", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,k,cols", SIZES)
def test_long_reductions_hold_fp32(rows, k, cols, xt, wt):
    require_gpu()
    from newton_schulz_11_b200 import api

    dt = {"f32": torch.float32, "bf16": torch.bfloat16}
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    a = torch.randn(rows, k, generator=gen, device="cuda").to(dt[xt])
    b = torch.randn(cols, k, generator=gen, device="cuda").to(dt[wt])
    want = a.double() @ b.double().t()
    piece = 512 if xt == wt == "bf16" else 256
    tol = piece / 16 * (2 / 3) * 2.0 ** -24 + (k / piece / 2) ** 0.5 * 2.0 ** -24

    def off(got):
        return float((got.double() - want).norm() / want.norm())

    none = torch.empty(0, device="cuda")
    y = api.linear(a, b, out=none.new_empty(rows, cols))
    # the same product as dx = dy w (w contiguous along its side) and as dw = dy^T x (both)
    bt = b.t().contiguous()
    dx = api.linear_backward(a, a.new_empty(rows, cols), bt, dx=none.new_empty(rows, cols), need_dw=False,
                             need_db=False)[0]
    dw = api.linear_backward(a.t().contiguous(), bt, b.new_empty(rows, cols), need_dx=False, need_db=False)[1]
    for name, got in (("y", y), ("dx", dx), ("dw", dw)):
        assert off(got) <= tol, (name, off(got), tol)
