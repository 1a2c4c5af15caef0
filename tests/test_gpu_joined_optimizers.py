"""A sharded step with an AdamW optimizer and an optimizer of whole matrices beside it: all three are applied or left
out as one, and a check that could no longer leave out what has been applied is refused.  Everything is compared bit for
bit, with the same steps made alone."""
import math

import pytest
import torch
from test_gpu_muon import Joined, Muon, stream

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
SIZES = [256, 1000, 7]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


class Tensors:
    """An AdamW optimizer of three tensors with fp32 gradients."""

    def __init__(self, seed=0):
        gen = torch.Generator().manual_seed(seed)
        new = lambda std: [(torch.randn(n, generator=gen) * std).cuda() for n in SIZES]  # noqa: E731
        self.p, self.g = new(0.02), new(1e-2)
        self.h = Z.zero_adamw_create(SIZES, 32, Z.ZERO_BF16, Z.ZERO_FP32)
        info = Z.zero_adamw_info(self.h)
        self.m, self.v, self.ws = (torch.zeros(max(16, n), dtype=torch.uint8, device="cuda")
                                   for n in (info.moment_bytes, info.moment_bytes, info.workspace_bytes))
        self.bind(0)

    def bind(self, t):
        Z.zero_adamw_bind(self.h, [t.data_ptr() for t in self.p], None, [t.data_ptr() for t in self.g],
                          self.m.data_ptr(), self.v.data_ptr(), None, self.ws.data_ptr(), t, stream())

    def state(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.p + [self.m, self.v]]

    def close(self):
        torch.cuda.synchronize()
        Z.zero_adamw_destroy(self.h)


class Three(Joined):
    def __init__(self):
        super().__init__(Z.scaler(scale=1.0))
        self.tensors = Tensors()
        self.ptrs = [c.data_ptr() for c in self.c]

    def matrices(self):
        torch.cuda.synchronize()
        return [t.clone() for t in self.mu.p + self.mu.p16 + self.mu.x]

    def plan(self):
        return [self.g.state_tensor(r, k).clone() for r in range(2) for k in ("master", "m", "v")]

    def close(self):
        self.tensors.close()
        super().close()


def refused(f, *args):
    with pytest.raises(Z.ZeroError) as e:
        f(*args)
    assert e.value.status == Z.ZERO_ESTATE, str(e.value)


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("first", ["tensors", "matrices"])
def test_all_are_applied_or_left_out(first, late):
    """Either order of the two parts; checks before the buckets, or (late) after them and before both parts."""
    j, alone, mat = Three(), Tensors(), Muon([(64, 96), (130, 40)], 2, "bf16").fill(8)
    h, muon, s = Z.hyper(), Z.muon_hyper(lr=0.01), stream()
    try:
        def step():
            checks = [lambda: Z.zero_adamw_check(j.tensors.h, j.g.plan, s), lambda: Z.zero_muon_check(j.mu.h, j.g.plan, muon, s)]
            parts = [lambda: Z.zero_adamw_step_with(j.tensors.h, j.g.plan, h, s),
                     lambda: Z.zero_muon_step_with(j.mu.h, j.g.plan, muon, s)]
            for calls in (checks, parts):
                if first == "matrices":
                    calls.reverse()
            for f in () if late else checks:
                f()
            Z.zero_step(j.g.plan, j.ptrs, -1, h, s)
            for f in (checks if late else []) + parts:
                f()
            return Z.zero_step_finish(j.g.plan, s)

        for t in (1, 2):
            assert step().skipped == 0
            Z.zero_adamw_step(alone.h, h, 1.0, s)
            Z.zero_muon_step(mat.h, muon, 1.0, s)
            assert all(torch.equal(a, b) for a, b in zip(alone.state(), j.tensors.state()))
            assert all(torch.equal(a, b) for a, b in zip(mat.p + mat.x, j.mu.p + j.mu.x))
        kept = j.plan() + j.tensors.state() + j.matrices()
        for spoil in (j.mu.g[1][0][5], j.tensors.g[1], j.c[1]):
            good = spoil[3].clone()
            spoil[3] = math.inf
            assert step().skipped == 1
            assert all(torch.equal(a, b) for a, b in zip(kept, j.plan() + j.tensors.state() + j.matrices()))
            spoil[3] = good
        assert step().t == 3 and Z.zero_muon_read(j.mu.h, s).t == 3 and Z.zero_adamw_read(j.tensors.h, s).t == 3
    finally:
        j.close()
        alone.close()
        mat.close()


@pytest.mark.parametrize("bad", [False, True])
def test_a_check_after_a_part_is_refused(bad):
    """What is moved could not be left out any more: the other optimizer's check, a second one's, and that of a handle
    whose bind or own step forgot its first check."""
    j, other, s = Three(), Tensors(1), stream()
    h, muon = Z.hyper(), Z.muon_hyper(lr=0.01)
    plan = j.g.plan
    try:
        def finish(t):
            res = Z.zero_step_finish(plan, s)
            assert res.skipped == 0 and res.t == t

        if bad:
            j.mu.g[0][1][2, 2] = math.inf
        Z.zero_adamw_check(j.tensors.h, plan, s)
        Z.zero_step(plan, j.ptrs, -1, h, s)
        Z.zero_adamw_step_with(j.tensors.h, plan, h, s)
        kept = j.matrices()
        refused(Z.zero_muon_check, j.mu.h, plan, muon, s)
        refused(Z.zero_muon_step_with, j.mu.h, plan, muon, s)
        refused(Z.zero_adamw_check, other.h, plan, s)
        finish(1)                                   # without the matrices
        assert all(torch.equal(a, b) for a, b in zip(kept, j.matrices()))
        j.mu.g[0][1][2, 2] = 0.0
        if bad:
            j.tensors.g[0][0] = math.nan
        Z.zero_muon_check(j.mu.h, plan, muon, s)
        Z.zero_step(plan, j.ptrs, -1, h, s)
        Z.zero_muon_step_with(j.mu.h, plan, muon, s)
        kept = j.tensors.state()
        refused(Z.zero_adamw_check, j.tensors.h, plan, s)
        refused(Z.zero_adamw_step_with, j.tensors.h, plan, h, s)
        for forget in (lambda: j.mu.bind(-1), lambda: Z.zero_muon_step(j.mu.h, muon, 1.0, s)):
            forget()
            refused(Z.zero_muon_check, j.mu.h, plan, muon, s)
            refused(Z.zero_muon_step_with, j.mu.h, plan, muon, s)
        finish(2)
        assert all(torch.equal(a, b) for a, b in zip(kept, j.tensors.state()))
        # the next step takes all of them again
        j.tensors.g[0][0] = 0.0
        Z.zero_muon_check(j.mu.h, plan, muon, s)
        Z.zero_adamw_check(j.tensors.h, plan, s)
        Z.zero_adamw_check(other.h, plan, s)
        Z.zero_step(plan, j.ptrs, -1, h, s)
        Z.zero_adamw_step_with(other.h, plan, h, s)
        Z.zero_muon_step_with(j.mu.h, plan, muon, s)
        Z.zero_adamw_step_with(j.tensors.h, plan, h, s)
        finish(3)
    finally:
        j.close()
        other.close()


def test_a_bind_after_the_check_is_another_check():
    """A bind may bring gradients that the check has not seen."""
    j, alone, h, s = Three(), Tensors(), Z.hyper(), stream()
    plan = j.g.plan
    try:
        Z.zero_adamw_check(j.tensors.h, plan, s)
        Z.zero_step(plan, j.ptrs, -1, h, s)
        j.tensors.bind(-1)
        refused(Z.zero_adamw_step_with, j.tensors.h, plan, h, s)
        Z.zero_adamw_check(j.tensors.h, plan, s)
        Z.zero_adamw_step_with(j.tensors.h, plan, h, s)
        j.tensors.bind(-1)
        refused(Z.zero_adamw_check, j.tensors.h, plan, s)
        refused(Z.zero_adamw_step_with, j.tensors.h, plan, h, s)
        assert Z.zero_step_finish(plan, s).t == 1
        Z.zero_adamw_step(alone.h, h, 1.0, s)
        assert all(torch.equal(a, b) for a, b in zip(alone.state(), j.tensors.state()))
    finally:
        j.close()
        alone.close()
