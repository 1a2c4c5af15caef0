"""zero_gated_backward where a factor leaves fp32's range and the gradient does not.

dg = dh u act'(g) is finite for every finite dh and u whose gradient is: where the slope is 0, so is dg, however large dh
and u are.  In bf16 their product reaches 1e76.  Sums of such columns and products with them are then those of zeros; the
values are whole powers of two elsewhere, so that everything compared is exact.
"""
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


@pytest.mark.parametrize("n", [64, 61])
@pytest.mark.parametrize("act,g", [(Z.ZERO_ACT_RELU, -1.0), (Z.ZERO_ACT_SILU, -512.0), (Z.ZERO_ACT_GELU_TANH, -64.0),
                                   (Z.ZERO_ACT_GELU, -64.0)])
def test_a_slope_of_zero_is_a_gradient_of_zero(act, g, n):
    m, k = 40, 32
    new = lambda r, c, v: torch.full((r, c), v, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    big = 2.0 ** 100
    x, wg, wu = new(m, k, 0.5), new(n, k, 0.25), new(n, k, 0.0)
    gate, up, dh = new(m, n, g), new(m, n, big), new(m, n, big)
    dx, dwg, dwu, dbg = new(m, k, 7.0), new(n, k, 7.0), new(n, k, 7.0), new(1, n, 7.0)
    args = Z.zero_gated_t(rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16, layout=Z.ZERO_WEIGHT_OUT_IN,
                          activation=act, x=x.data_ptr(), w_gate=wg.data_ptr(), w_up=wu.data_ptr(), gate=gate.data_ptr(),
                          up=up.data_ptr(), dh=dh.data_ptr(), dx=dx.data_ptr(), dw_gate=dwg.data_ptr(),
                          dw_up=dwu.data_ptr(), db_gate=dbg.data_ptr())
    size = Z.zero_gated_workspace(args, True)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    Z.zero_gated_backward(args, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    # act(g) is 0 there too, but for the sign
    for name, v in (("dx", dx), ("dw_gate", dwg), ("dw_up", dwu), ("db_gate", dbg)):
        assert not bool(v.any()), (name, float(v.flatten()[0]))


def test_a_product_beyond_the_range_times_a_small_slope():
    """2^100 * 2^60 * silu'(-80): 2^160 is out of range, the gradient is about -1e14."""
    m, k, n = 8, 16, 16
    new = lambda r, c, v: torch.full((r, c), v, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    gate, up, dh, x, w, dw = new(m, n, -80.0), new(m, n, 2.0 ** 60), new(m, n, 2.0 ** 100), new(m, k, 1.0), new(n, k, 0.0), new(n, k, 0.0)
    args = Z.zero_gated_t(rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16, layout=Z.ZERO_WEIGHT_OUT_IN,
                          activation=Z.ZERO_ACT_SILU, x=x.data_ptr(), gate=gate.data_ptr(), up=up.data_ptr(),
                          dh=dh.data_ptr(), dw_gate=dw.data_ptr())
    size = Z.zero_gated_workspace(args, True)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    Z.zero_gated_backward(args, ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    z = torch.tensor(-80.0, dtype=torch.float64)
    s = torch.sigmoid(z)
    want = m * 2.0 ** 160 * float(s * (1 + z * (1 - s)))
    # dg's rounding and the result's, 2^-8 each; the slope's: 2^-17 of the terms, here 80 e^-80 and less
    assert bool(((dw.double() - want).abs() <= (2.0 ** -7 + 2.0 ** -14) * abs(want)).all()), (float(dw[0, 0]), want)
