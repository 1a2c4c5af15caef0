"""zero_muon's host side (no GPU): sizes, refusals, and the order of its kernels."""
import pytest
from test_operators_order_host import source, test_every_kernel_waits_for_itself

import zero_sharded_mixed_03_gb300 as Z


def refused(status, f, *args, **kw):
    with pytest.raises(Z.ZeroError) as e:
        f(*args, **kw)
    assert e.value.status == status, str(e.value)


def test_create():
    for rows, cols, n_d, kind in (([-1], [4], 1, 0), ([4], [-1], 1, 0), ([4], [4], 0, 0), ([4], [4], 1, 2)):
        refused(Z.ZERO_EINVAL, Z.zero_muon_create, rows, cols, n_d, kind)
    for rows, cols, n_d in (([Z.ZERO_MUON_MAX_SIZE + 1], [1], 1), ([1], [Z.ZERO_MUON_MAX_SIZE + 1], 1),
                            ([Z.ZERO_MUON_MAX_SIDE + 1], [Z.ZERO_MUON_MAX_SIDE + 1], 1), ([4], [4], 129),
                            ([1] * (Z.ZERO_MUON_MAX_MATRICES + 1), [1] * (Z.ZERO_MUON_MAX_MATRICES + 1), 1)):
        refused(Z.ZERO_ERANGE, Z.zero_muon_create, rows, cols, n_d)
    with pytest.raises(ValueError):
        Z.zero_muon_create([1, 2], [1])
    Z.zero_muon_destroy(0)


def test_info():
    h = Z.zero_muon_create([3, 0, 100, 64], [5, 7, 30, 64], 2)
    try:
        info = Z.zero_muon_info(h)
        assert (info.n_matrices, info.n_contribs, info.elems) == (4, 2, 15 + 3000 + 4096)
        assert info.state_elems == 256 + 3072 * 1 + 4096          # 15, 3000 and 4096 rounded up to 256
        # three buffers of each X and two of each smaller side's square, 16 bits
        assert info.workspace_bytes >= 2 * (3 * (3000 + 4096) + 2 * (30 * 32 + 4096))
    finally:
        Z.zero_muon_destroy(h)
    h = Z.zero_muon_create([], [])
    assert Z.zero_muon_info(h).elems == 0
    Z.zero_muon_destroy(h)


def test_bind_refusals():
    h = Z.zero_muon_create([8, 0], [16, 3], 2)
    good = dict(params=[4096, None], params16=[8192, None], updates=[16384, None], grads=[32768, 0, 65536, 0],
                momentum=[1 << 17, 1 << 18], workspace=1 << 19)
    try:
        for status, change in ((Z.ZERO_EINVAL, dict(workspace=0)), (Z.ZERO_EALIGN, dict(workspace=(1 << 19) + 16)),
                               (Z.ZERO_EINVAL, dict(t=-1)), (Z.ZERO_EINVAL, dict(t=-2)),
                               (Z.ZERO_EINVAL, dict(momentum=[1 << 17, 0])),
                               (Z.ZERO_EINVAL, dict(momentum=[1 << 17, 1 << 17])),
                               (Z.ZERO_EALIGN, dict(momentum=[(1 << 17) + 4, 1 << 18])),
                               (Z.ZERO_EINVAL, dict(grads=[32768, 0, None, 0])),
                               (Z.ZERO_EALIGN, dict(grads=[32768, 0, 65537, 0])),
                               (Z.ZERO_EALIGN, dict(params=[4098, None])), (Z.ZERO_EALIGN, dict(params16=[8193, None])),
                               (Z.ZERO_EALIGN, dict(updates=[8193, None])),
                               (Z.ZERO_EINVAL, dict(params=None)), (Z.ZERO_EINVAL, dict(params=None, params16=None, updates=None))):
            refused(status, Z.zero_muon_bind, h, **{**good, **change})
        for change in (dict(params=[4096]), dict(grads=[32768, 0]), dict(momentum=[1 << 17])):
            with pytest.raises(ValueError):
                Z.zero_muon_bind(h, **{**good, **change})
        refused(Z.ZERO_EINVAL, lambda: Z._check(Z.lib().zero_muon_bind(None, *[None] * 6, 0, None)))
    finally:
        Z.zero_muon_destroy(h)


def test_step_refusals():
    h, plan = Z.zero_muon_create([8], [16]), Z.zero_plan_create([64], 2, 2, 0, None, Z.ZERO_BF16)
    try:
        refused(Z.ZERO_ESTATE, Z.zero_muon_step, h, Z.muon_hyper())          # nothing bound
        refused(Z.ZERO_EINVAL, Z.zero_muon_step, 0, Z.muon_hyper())
        refused(Z.ZERO_ESTATE, Z.zero_muon_read, h)
        for scale in (0.0, -1.0, float("inf"), float("nan")):
            refused(Z.ZERO_EINVAL, Z.zero_muon_step, h, Z.muon_hyper(), scale)
        nan = float("nan")
        bad = [dict(momentum=1.0), dict(momentum=-0.1), dict(momentum=nan), dict(lr=nan), dict(eps=0.0), dict(eps=nan),
               dict(weight_decay=float("inf")), dict(steps=0), dict(steps=9, coefficients=[(1, 0, 0)] * 9), dict(scale=3),
               dict(scale=-1), dict(coefficients=(nan, 0, 0))]
        for change in bad:
            hyper = Z.muon_hyper(**change)
            refused(Z.ZERO_EINVAL, Z.zero_muon_step, h, hyper)
            refused(Z.ZERO_EINVAL, Z.zero_muon_check, h, plan, hyper)
            refused(Z.ZERO_EINVAL, Z.zero_muon_step_with, h, plan, hyper)
        # singular values of 1 may grow to 3, 9, 27
        refused(Z.ZERO_ERANGE, Z.zero_muon_step, h, Z.muon_hyper(steps=3, coefficients=(3.0, 0.0, 0.0)))
        refused(Z.ZERO_ESTATE, Z.zero_muon_step, h, Z.muon_hyper(steps=1, coefficients=(3.0, 0.0, 0.0)))
        refused(Z.ZERO_ESTATE, Z.zero_muon_step, h, Z.muon_hyper(steps=8))
        hyper = Z.muon_hyper()
        hyper.flags = 2
        refused(Z.ZERO_EINVAL, Z.zero_muon_step, h, hyper)
        refused(Z.ZERO_EINVAL, Z.zero_muon_check, h, 0, Z.muon_hyper())
        refused(Z.ZERO_EINVAL, Z.zero_muon_check, 0, plan, Z.muon_hyper())
        refused(Z.ZERO_ESTATE, Z.zero_muon_check, h, plan, Z.muon_hyper())
        refused(Z.ZERO_ESTATE, Z.zero_muon_step_with, h, plan, Z.muon_hyper())
        with pytest.raises(ValueError):
            Z.muon_hyper(steps=5, coefficients=[(1, 0, 0)] * 4)
    finally:
        Z.zero_muon_destroy(h)
        Z.zero_plan_destroy(plan)


def test_order():
    test_every_kernel_waits_for_itself("zero_muon.cu")
    assert not any(w in source("zero_muon.cu") for w in ("griddepcontrol", "__ldg", "ld.global.nc", "__restrict__"))
