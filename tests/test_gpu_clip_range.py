"""A clipped sharded step whose finite gradients have squares beyond fp32's range.

The norm is infinite and the coefficient 0 (the rule's oracle: norm^2 is the sum in double of fp32 squares): the
step is applied with gradients of 0, nothing becomes not a number, and the next step is an ordinary one.
"""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z
from zero_sharded_mixed_03_gb300.emulate import EmulatedGroup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()


@pytest.mark.parametrize("n", [3000, 100_001])
@pytest.mark.parametrize("staging", [Z.ZERO_STAGING_REGISTER_LOADS, Z.ZERO_STAGING_BULK, None])
@pytest.mark.parametrize("at", [0, 1711, 2999])
def test_infinite_norm_of_finite_gradients(n, staging, at):
    """staging None: offloaded to host threads."""
    n_d = 4
    g = EmulatedGroup([n], n_d, 2, offload=staging is None, offload_threads=2 if staging is None else 0)
    try:
        if staging is not None:
            g.set_option(Z.ZERO_OPT_STAGING, staging)
        gen = torch.Generator().manual_seed(1)
        for r in range(n_d):
            for _u, off, k, _b, _s in g.shard_slices(r):
                g.state[r]["master"][0][off:off + k] = torch.randn(k, generator=gen) * 0.02
        contribs = [torch.zeros(int(g.info.max_contrib_elems), dtype=torch.bfloat16, device="cuda") for _ in range(n_d)]
        for c in contribs:
            c[:n] = (torch.randn(n, generator=gen) * 1e-2).to(torch.bfloat16).cuda()
        kept = contribs[2][at].clone()
        contribs[2][at] = 1e25
        h = Z.hyper(max_grad_norm=1.0)
        before = [g.state_tensor(r, "master").clone() for r in range(n_d)]

        def step():
            g.grad_norm([c.data_ptr() for c in contribs], -1)
            g.step([c.data_ptr() for c in contribs], -1, h)
            return g.finish()

        res = step()
        assert res.skipped == 0 and res.t == 1 and res.grad_norm == math.inf
        decay = np.float32(h.lr * h.weight_decay)
        for r in range(n_d):
            p = before[r].cpu().numpy()
            assert np.array_equal(g.state_tensor(r, "master").cpu().numpy(), p - decay * p)
            assert not g.state_tensor(r, "m").any() and not g.state_tensor(r, "v").any()
        contribs[2][at] = kept
        res = step()
        assert res.skipped == 0 and res.t == 2 and 0.0 < res.grad_norm < 10.0
        for r in range(n_d):
            assert bool(torch.isfinite(g.state_tensor(r, "master")).all())
    finally:
        torch.cuda.synchronize()
        g.close()
