"""Refusals of zero_adamw_check and zero_adamw_step_with (no GPU)."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def refused(status, f, *args):
    with pytest.raises(Z.ZeroError) as e:
        f(*args)
    assert e.value.status == status and e.value.args


def test_refusals():
    plan, h = Z.zero_plan_create([64], 2, 2, 0, None, Z.ZERO_BF16), Z.zero_adamw_create([100], 8)
    try:
        refused(Z.ZERO_EINVAL, Z.zero_adamw_check, h, 0)
        refused(Z.ZERO_EINVAL, Z.zero_adamw_check, 0, plan)
        refused(Z.ZERO_ESTATE, Z.zero_adamw_check, h, plan)                 # nothing bound
        refused(Z.ZERO_EINVAL, Z.zero_adamw_step_with, h, 0, Z.hyper())
        refused(Z.ZERO_EINVAL, Z.zero_adamw_step_with, 0, plan, Z.hyper())
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, h, plan, Z.hyper())
        for hyper in (Z.hyper(beta1=1.0), Z.hyper(eps=-1.0), Z.hyper(max_grad_norm=float("nan"))):
            refused(Z.ZERO_EINVAL, Z.zero_adamw_step_with, h, plan, hyper)
    finally:
        Z.zero_adamw_destroy(h)
        Z.zero_plan_destroy(plan)
