"""zero_adamw's host side (no GPU): layout sizes and refusals."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def refused(status, f, *args):
    with pytest.raises(Z.ZeroError) as e:
        f(*args)
    assert e.value.status == status and e.value.args


def test_layout():
    for bits in (8, 32):
        h = Z.zero_adamw_create([0, 1, 256, 257], bits, Z.ZERO_FP16, Z.ZERO_FP32)
        info = Z.zero_adamw_info(h)
        assert (info.n_tensors, info.elems, info.n_blocks, info.state_elems) == (4, 514, 4, 1024)
        assert info.moment_bytes == 1024 * bits // 8 and info.scale_bytes == (8 if bits == 8 else 0)
        assert info.workspace_bytes >= 256 + 4 * 40 + 4 * 4
        Z.zero_adamw_destroy(h)
    Z.zero_adamw_destroy(0)


def test_create_refusals():
    for args in (([4], 16, Z.ZERO_BF16, Z.ZERO_BF16), ([4], 8, Z.ZERO_FP32, Z.ZERO_BF16), ([4], 8, Z.ZERO_BF16, 3),
                 ([-1], 8, Z.ZERO_BF16, Z.ZERO_BF16)):
        refused(Z.ZERO_EINVAL, Z.zero_adamw_create, *args)
    refused(Z.ZERO_ERANGE, Z.zero_adamw_create, [1 << 41], 8)
    refused(Z.ZERO_ERANGE, Z.zero_adamw_create, [1 << 37] * 3, 8)


def test_bind_and_step_refusals():
    h = Z.zero_adamw_create([100, 0], 8)
    try:
        ok = dict(params=[4096, 0], params16=[8192, 0], grads=[16384, 0], m=256, v=512, scales=1024, workspace=2048, t=0)

        def bind(status, **change):
            refused(status, lambda: Z.zero_adamw_bind(h, **{**ok, **change}))

        bind(Z.ZERO_EINVAL, params=[0, 0])
        bind(Z.ZERO_EINVAL, grads=[0, 0])
        bind(Z.ZERO_EINVAL, m=0)
        bind(Z.ZERO_EINVAL, v=0)
        bind(Z.ZERO_EINVAL, scales=0)
        bind(Z.ZERO_EINVAL, workspace=0)
        bind(Z.ZERO_EINVAL, t=-1)
        bind(Z.ZERO_EINVAL, t=-2)
        bind(Z.ZERO_EALIGN, params=[4098, 0])
        bind(Z.ZERO_EALIGN, params16=[8193, 0])
        bind(Z.ZERO_EALIGN, grads=[16385, 0])
        bind(Z.ZERO_EALIGN, m=264)
        bind(Z.ZERO_EALIGN, scales=1025)
        bind(Z.ZERO_EALIGN, workspace=2056)
        with pytest.raises(ValueError):
            Z.zero_adamw_bind(h, **{**ok, "grads": [16384]})
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step, h, Z.hyper())
        refused(Z.ZERO_ESTATE, Z.zero_adamw_read, h)
        refused(Z.ZERO_ESTATE, Z.zero_adamw_export, h, 256, 512)
        refused(Z.ZERO_EALIGN, Z.zero_adamw_export, h, 257, 512)
        refused(Z.ZERO_EINVAL, Z.zero_adamw_export, h, 0, 512)
        for hyper in (Z.hyper(beta1=1.0), Z.hyper(beta2=-0.1), Z.hyper(eps=-1.0), Z.hyper(lr=float("nan")),
                      Z.hyper(max_grad_norm=float("nan"))):
            refused(Z.ZERO_EINVAL, Z.zero_adamw_step, h, hyper)
        for scale in (0.0, -1.0, float("inf"), float("nan")):
            refused(Z.ZERO_EINVAL, Z.zero_adamw_step, h, Z.hyper(), scale)
    finally:
        Z.zero_adamw_destroy(h)
    h = Z.zero_adamw_create([100], 32)
    refused(Z.ZERO_EINVAL, Z.zero_adamw_export, h, 256, 512)
    Z.zero_adamw_destroy(h)
