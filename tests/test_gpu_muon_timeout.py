"""zero_muon's products give up waiting for one another: the status that the host reads, and what the step then counts as.

With the limit 0 a block looks a few times for the product before, which here takes at least 50 us, and gives up; every
kernel ends by itself.  Nothing is compared but what such a step leaves alone and the steps after it, bit for bit.
"""
import pytest
import torch
from test_gpu_joined_step import Both
from test_gpu_muon import Joined, Muon, stream

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
USUAL = 2_000_000_000
# a product on blocks of their own, and on pairs of them
SHAPES = [[(256, 65536)], [(2048, 8192), (2048, 8192)]]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def timed_out(f, *args):
    with pytest.raises(Z.ZeroError) as e:
        f(*args)
    assert e.value.status == Z.ZERO_ETIMEOUT, str(e.value)
    return e.value.result


def limit(mu, ns):
    Z.zero_muon_set_option(mu.h, Z.ZERO_MUON_OPT_WAIT_LIMIT_NS, ns)


def restore(mu, saved):
    for v, old in zip(mu.p + mu.p16 + mu.x, saved):
        v.copy_(old)


@pytest.mark.parametrize("shapes", SHAPES)
def test_a_step_of_its_own(shapes):
    mu, ref, hyper, s = Muon(shapes).fill(1), Muon(shapes).fill(1), Z.muon_hyper(lr=0.01), stream()
    try:
        assert mu.step(hyper).t == ref.step(hyper).t == 1
        saved = [v.clone() for v in mu.p + mu.p16 + mu.x]
        half = mu.halves[1].clone()
        limit(mu, 0)
        Z.zero_muon_step(mu.h, hyper, 1.0, s)
        torch.cuda.synchronize()
        limit(mu, USUAL)
        restore(mu, saved)
        Z.zero_muon_step(mu.h, hyper, 1.0, s)            # left out: the one before is not read yet
        assert all(torch.equal(a, b) for a, b in zip(saved, mu.p + mu.p16 + mu.x))
        res = timed_out(Z.zero_muon_read, mu.h, s)
        assert (res.t, res.skipped, res.skipped_total, res.finished, res.current) == (1, 1, 2, 3, 1)
        assert torch.equal(half, mu.halves[1])
        timed_out(Z.zero_operators_check, s)
        assert Z.zero_muon_read(mu.h, s).t == 1          # told once
        assert mu.step(hyper).t == ref.step(hyper).t == 2
        assert all(torch.equal(a, b) for a, b in zip(ref.p + ref.x + ref.halves, mu.p + mu.x + mu.halves))
        mu.guards_stand()
    finally:
        mu.close()
        ref.close()


@pytest.mark.parametrize("shapes", SHAPES)
def test_a_part_of_a_sharded_step(shapes):
    j, ref = Joined(Z.scaler(scale=1.0)), Joined(Z.scaler(scale=1.0))
    hyper, muon, s = Z.hyper(), Z.muon_hyper(lr=0.01), stream()
    for b in (j, ref):
        b.mu.close()
        b.mu = Muon(shapes, 2).fill(1)
    try:
        assert j.step(hyper, muon).t == ref.step(hyper, muon).t == 1
        saved = [v.clone() for v in j.mu.p + j.mu.p16 + j.mu.x]
        plan = [j.g.state_tensor(r, k).clone() for r in range(2) for k in ("master", "m", "v")] + [j.g.full16.clone()]
        limit(j.mu, 0)
        res = timed_out(j.step, hyper, muon)
        assert (res.t, res.skipped, res.finished) == (1, 1, 1)
        assert all(torch.equal(a, b) for a, b in
                   zip(plan, [j.g.state_tensor(r, k) for r in range(2) for k in ("master", "m", "v")] + [j.g.full16]))
        limit(j.mu, USUAL)
        restore(j.mu, saved)
        res = timed_out(Z.zero_muon_read, j.mu.h, s)
        assert (res.t, res.skipped, res.current) == (1, 1, 1)
        timed_out(Z.zero_operators_check, s)
        assert j.step(hyper, muon).t == ref.step(hyper, muon).t == 2
        assert all(torch.equal(a, b) for a, b in zip(ref.mu.p + ref.mu.halves, j.mu.p + j.mu.halves))
        assert torch.equal(j.g.full16, ref.g.full16)
    finally:
        j.close()
        ref.close()


def test_a_part_of_an_offloaded_step():
    """The host's update waits for the matrices' products: a step that they discard leaves the host's state alone."""
    both, ref, mu = Both(offload=True), Both(offload=True), Muon(SHAPES[0]).fill(1)
    hyper, muon, s = Z.hyper(), Z.muon_hyper(lr=0.01), stream()

    def step(b, with_matrices):
        contribs = [[c.data_ptr() for c in unit] for unit in b.c]
        if with_matrices:
            Z.zero_muon_check(mu.h, b.g.plan, muon, s)
        for i, which in enumerate(b.calls):
            b.g.step(contribs[i], which, hyper)
        if with_matrices:
            Z.zero_muon_step_with(mu.h, b.g.plan, muon, s)
        return b.g.finish()

    try:
        for b in (both, ref):
            b.gradients(1)
        assert step(both, True).t == step(ref, False).t == 1
        assert all(torch.equal(a, b) for a, b in zip(both.state(), ref.state()))
        limit(mu, 0)
        both.gradients(2)
        assert timed_out(step, both, True).t == 1
        assert all(torch.equal(a, b) for a, b in zip(both.state(), ref.state()))
        limit(mu, USUAL)
        timed_out(Z.zero_muon_read, mu.h, s)
        timed_out(Z.zero_operators_check, s)
        for b in (both, ref):
            b.gradients(3)
        assert step(both, True).t == step(ref, False).t == 2
        assert all(torch.equal(a, b) for a, b in zip(both.state(), ref.state()))
    finally:
        mu.close()
        both.close()
        ref.close()
