"""zero_block_norm's host side (no GPU): workspace sizes and refusals."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def args(**change):
    base = dict(rows=32, dim=64, dtype16=Z.ZERO_BF16, kind=Z.ZERO_NORM_RMS, norms=Z.ZERO_NORM_PRE | Z.ZERO_NORM_POST,
                rows_per_gate=4, eps=1e-5, residual_scale=1.0)
    names = ("h", "x", "gate", "y", "z", "dy", "dz", "dx", "dh", "dgate", "dpost_w", "dpre_w")
    base.update({name: 4096 * (i + 1) for i, name in enumerate(names)})
    base.update(change)
    return Z.zero_block_norm_t(**base)


def refused(status, back, **change):
    a = args(**change)
    calls = [lambda: Z.zero_block_norm_backward(a, 0, 0), lambda: Z.zero_block_norm_workspace(a)] if back else [lambda: Z.zero_block_norm(a)]
    for f in calls:
        with pytest.raises(Z.ZeroError) as e:
            f()
        assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("back", [False, True])
def test_refusals(back):
    for change in (dict(rows=-1), dict(dim=0), dict(dtype16=2), dict(kind=2), dict(norms=4), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(residual_scale=float("inf")), dict(rows_per_gate=0), dict(gate=None),
                   dict(rows_per_gate=-1), dict(ld_h=63), dict(ld_dx=1)):
        refused(Z.ZERO_EINVAL, back, **change)
    for change in (dict(dim=Z.ZERO_NORM_MAX_DIM + 1), dict(rows=1 << 41), dict(ld_y=1 << 40)):
        refused(Z.ZERO_ERANGE, back, **change)
    for name in ("h", "x", "gate", "y", "z", "dy", "dz", "dx", "dh", "dgate", "dpost_w", "dpre_w", "post_w", "pre_b"):
        refused(Z.ZERO_EALIGN, back, **{name: 4097})


def test_forward_refusals():
    for change in (dict(h=None), dict(z=None), dict(norms=0, y=None), dict(y=4096), dict(y=8192, ld_y=72), dict(z=4096, ld_z=72),
                   dict(z=8192)):
        refused(Z.ZERO_EINVAL, False, **change)


def test_backward_refusals():
    for change in (dict(h=None), dict(y=None), dict(dz=None), dict(norms=Z.ZERO_NORM_POST), dict(norms=Z.ZERO_NORM_PRE),
                   dict(gate=None, rows_per_gate=0),
                   dict(dx=None, dh=None, dgate=None, dpost_w=None, dpre_w=None), dict(dx=7 * 4096), dict(dx=6 * 4096, ld_dx=72)):
        refused(Z.ZERO_EINVAL, True, **change)
    a = args()
    n = Z.zero_block_norm_workspace(a)
    assert n > 0
    for ws, size, status in ((0, n, Z.ZERO_EINVAL), (8, n, Z.ZERO_EALIGN), (256, n - 1, Z.ZERO_ERANGE)):
        with pytest.raises(Z.ZeroError) as e:
            Z.zero_block_norm_backward(a, ws, size)
        assert e.value.status == status
    assert Z.zero_block_norm_workspace(args(dgate=None, dpost_w=None, dpre_w=None)) == 0
