"""zero_linear's host side (no GPU): workspace sizes and refusals."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def args(**change):
    base = dict(rows=32, in_features=64, out_features=128, dtype16=Z.ZERO_BF16, layout=Z.ZERO_WEIGHT_OUT_IN,
                activation=Z.ZERO_ACT_NONE, x=4096, w=8192, y=16384, dy=32768, dx=65536, dw=131072)
    base.update(change)
    return Z.zero_linear_t(**base)


def refused(status, back, **change):
    a = args(**change)
    call = Z.zero_linear_backward if back else Z.zero_linear
    for f in (lambda: Z.zero_linear_workspace(a, back), lambda: call(a, 0, 0)):
        with pytest.raises(Z.ZeroError) as e:
            f()
        assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("back", [False, True])
def test_refusals(back):
    for change in (dict(rows=-1), dict(in_features=-1), dict(out_features=-1), dict(dtype16=2), dict(layout=2),
                   dict(activation=5), dict(activation=-1), dict(flags=2), dict(ld_x=63), dict(ld_w=63), dict(ld_dy=127),
                   dict(x=None), dict(w=None)):
        refused(Z.ZERO_EINVAL, back, **change)
    for change in (dict(rows=1 << 31), dict(in_features=(1 << 30) + 1), dict(ld_x=1 << 40)):
        refused(Z.ZERO_ERANGE, back, **change)
    for name in ("x", "w", "y", "dy", "dx", "dw", "bias", "residual", "pre", "dbias"):
        refused(Z.ZERO_EALIGN, back, **{name: 4097})


def test_forward_refusals():
    refused(Z.ZERO_EINVAL, False, y=None)
    refused(Z.ZERO_EINVAL, False, flags=Z.ZERO_LINEAR_ACCUMULATE)
    refused(Z.ZERO_EINVAL, False, pre=16384)
    refused(Z.ZERO_EINVAL, False, residual=16384, ld_residual=136)


def test_backward_refusals():
    refused(Z.ZERO_EINVAL, True, dy=None)
    refused(Z.ZERO_EINVAL, True, dx=None, dw=None)
    refused(Z.ZERO_EINVAL, True, activation=Z.ZERO_ACT_SILU)


def test_workspace():
    # rows that do not start on 16 bytes are copied: 2 bytes an element, rows rounded up to 8
    plain, odd = Z.zero_linear_workspace(args()), Z.zero_linear_workspace(args(x=4098))
    assert odd - plain >= 2 * 32 * 64
    assert Z.zero_linear_workspace(args(activation=Z.ZERO_ACT_SILU, pre=4096), True) >= 2 * 32 * 128
    big = args(rows=8192, in_features=2048, out_features=8192)
    assert Z.zero_linear_workspace(big) == 0
    a = args(x=4098)
    for ws, n, status in ((0, odd, Z.ZERO_EINVAL), (8, odd, Z.ZERO_EALIGN), (256, odd - 1, Z.ZERO_ERANGE)):
        with pytest.raises(Z.ZeroError) as e:
            Z.zero_linear(a, ws, n)
        assert e.value.status == status
