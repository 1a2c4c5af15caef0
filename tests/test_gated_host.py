"""zero_gated's host side (no GPU): workspace sizes, refusals, and the order of its kernels."""
import pytest
from test_operators_order_host import source, test_every_kernel_waits_for_itself

import zero_sharded_mixed_03_gb300 as Z


def args(**change):
    base = dict(rows=32, in_features=64, out_features=128, dtype16=Z.ZERO_BF16, layout=Z.ZERO_WEIGHT_OUT_IN,
                activation=Z.ZERO_ACT_SILU, x=4096, w_gate=8192, w_up=16384, h=32768, gate=65536, up=1 << 17,
                dh=1 << 18, dx=1 << 19, dw_gate=1 << 20, dw_up=1 << 21, db_gate=1 << 22, db_up=1 << 23)
    base.update(change)
    return Z.zero_gated_t(**base)


def refused(status, back, **change):
    a = args(**change)
    call = Z.zero_gated_backward if back else Z.zero_gated
    for f in (lambda: Z.zero_gated_workspace(a, back), lambda: call(a, 0, 0)):
        with pytest.raises(Z.ZeroError) as e:
            f()
        assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("back", [False, True])
def test_refusals(back):
    for change in (dict(rows=-1), dict(in_features=-1), dict(out_features=-1), dict(dtype16=2), dict(layout=2),
                   dict(activation=5), dict(activation=-1), dict(flags=2), dict(ld_x=63), dict(ld_w_gate=63),
                   dict(ld_w_up=63), dict(ld_h=127), dict(ld_gate=127), dict(ld_dh=1), dict(ld_dw_up=63),
                   dict(x=None), dict(w_gate=None), dict(w_up=None)):
        refused(Z.ZERO_EINVAL, back, **change)
    for change in (dict(rows=1 << 31), dict(in_features=(1 << 30) + 1), dict(out_features=1 << 40), dict(ld_x=1 << 40)):
        refused(Z.ZERO_ERANGE, back, **change)
    for name in ("x", "w_gate", "w_up", "b_gate", "b_up", "h", "gate", "up", "dh", "dx", "dw_gate", "dw_up",
                 "db_gate", "db_up"):
        refused(Z.ZERO_EALIGN, back, **{name: 4097})
    with pytest.raises(Z.ZeroError):
        Z.lib() and Z._check(Z.lib().zero_gated_workspace(None, 0, None))


def test_forward_refusals():
    refused(Z.ZERO_EINVAL, False, h=None)
    refused(Z.ZERO_EINVAL, False, flags=Z.ZERO_GATED_ACCUMULATE)
    refused(Z.ZERO_EINVAL, False, gate=32768)
    refused(Z.ZERO_EINVAL, False, up=32768)
    refused(Z.ZERO_EINVAL, False, gate=1 << 17)


def test_backward_refusals():
    for name in ("dh", "gate", "up"):
        refused(Z.ZERO_EINVAL, True, **{name: None})
    refused(Z.ZERO_EINVAL, True, dx=None, dw_gate=None, dw_up=None, db_gate=None, db_up=None)
    refused(Z.ZERO_EINVAL, True, dw_gate=1 << 21)
    refused(Z.ZERO_EINVAL, True, db_gate=1 << 23)


@pytest.mark.timeout(20)
@pytest.mark.parametrize("back", [False, True])
def test_largest_sizes_are_laid_out_at_once(back):
    """A size is refused where its matrices are beyond any memory, and the tiles of the largest are dealt without
    looking at every way."""
    refused(Z.ZERO_ERANGE, back, rows=1 << 30, in_features=1 << 30, out_features=1 << 30)
    refused(Z.ZERO_ERANGE, back, rows=1, in_features=1 << 30, out_features=1 << 13)
    large = args(rows=1 << 20, in_features=1 << 21, out_features=1 << 21)
    # dg and du are 2^41 elements each
    assert Z.zero_gated_workspace(large, back) >= (2 * 2 * (1 << 41) if back else 0)


def test_workspace():
    assert Z.zero_gated_workspace(args()) == 0
    # rows that do not start on 16 bytes are copied: 2 bytes an element, rows rounded up to 8
    assert Z.zero_gated_workspace(args(x=4098)) >= 2 * 32 * 64
    assert Z.zero_gated_workspace(args(w_gate=8194, w_up=16386)) >= 2 * 2 * 64 * 128
    # one and two rows are read where they lie
    assert Z.zero_gated_workspace(args(rows=2)) == 0
    # dg and du; the sums where a bias wants them
    plain, none = Z.zero_gated_workspace(args(), True), Z.zero_gated_workspace(args(db_gate=None, db_up=None), True)
    assert plain > none >= 2 * 2 * 32 * 128
    assert Z.zero_gated_workspace(args(dx=None, dw_gate=None, dw_up=None), True) < plain
    a = args(x=4098)
    n = Z.zero_gated_workspace(a)
    for ws, size, status in ((0, n, Z.ZERO_EINVAL), (8, n, Z.ZERO_EALIGN), (256, n - 1, Z.ZERO_ERANGE)):
        with pytest.raises(Z.ZeroError) as e:
            Z.zero_gated(a, ws, size)
        assert e.value.status == status


def test_order():
    test_every_kernel_waits_for_itself("zero_gated.cu")
    for name in ("zero_gated.cu", "zero_mma.cuh"):
        assert not any(w in source(name) for w in ("griddepcontrol", "__ldg", "ld.global.nc", "__restrict__"))
