"""zero_adamw_check / zero_adamw_step_with: one step of a sharded plan and of separately held tensors.

Applied or left out as one, unscaled by the plan's loss scale, clipped by the norm of all gradients.  A clipped
step is compared with float64 AdamW over all parameters together.  Tolerances: as in
test_gpu_adamw.py, u = 2^-24 a rounding; the gradient has up to 8 (the ranks' mean, unscaling, the coefficient and the
norm behind it), so 12 u of each moment's terms, twice that for v.
"""
import math

import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z
from zero_sharded_mixed_03_gb300.emulate import EmulatedGroup

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SHARDED = [4096, 300, 1024, 77]              # two units of stage 3
REST = [256, 1000, 7, 513]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def stream():
    return torch.cuda.current_stream().cuda_stream


class Both:
    """A plan (stage 3 in two units, or stage 2 in one bucket) and an optimizer of the tensors that it leaves out."""

    def __init__(self, stage=3, bits=32, n_d=2, grad="fp32", offload=False, seed=0):
        self.n_d, self.bits, self.offload = n_d, bits, offload
        kw = dict(unit_first=[0, 2]) if stage == 3 else {}
        self.g = EmulatedGroup(SHARDED, n_d, stage, offload=offload, offload_threads=2 if offload else 0, **kw)
        self.calls = list(range(2)) if stage == 3 else [-1]
        gen = torch.Generator().manual_seed(seed)
        for r in range(n_d):
            for _u, off, n, _b, _s in self.g.shard_slices(r):
                part = (torch.randn(n, generator=gen) * 0.02).to(torch.bfloat16)
                self.g.state[r]["master"][0][off:off + n] = part.float()
                out = self.g.shard16[r] if stage == 3 else self.g.full16
                at = off if stage == 3 else r * n
                out[at:at + n] = part.cuda().view(torch.int16)
        n = int(self.g.info.max_contrib_elems)
        self.c = [[torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(n_d)] for _ in self.calls]
        self.offs, at = [], 3
        for size in REST:
            self.offs.append(at)
            at += size + 5
        gt, kind = {"fp32": (torch.float32, Z.ZERO_FP32), "bf16": (torch.bfloat16, Z.ZERO_BF16)}[grad]
        self.p = (torch.randn(at, generator=gen) * 0.02).cuda()
        self.p16 = self.p.to(torch.bfloat16)
        self.rest = torch.zeros(at, dtype=gt, device="cuda")
        self.h = Z.zero_adamw_create(REST, bits, Z.ZERO_BF16, kind)
        info = Z.zero_adamw_info(self.h)
        self.buf = [torch.zeros(max(16, k), dtype=torch.uint8, device="cuda")
                    for k in (info.moment_bytes, info.moment_bytes, info.scale_bytes, info.workspace_bytes)]
        ptrs = [[t.data_ptr() + o * t.element_size() for o in self.offs] for t in (self.p, self.p16, self.rest)]
        Z.zero_adamw_bind(self.h, *ptrs, self.buf[0].data_ptr(), self.buf[1].data_ptr(),
                          self.buf[2].data_ptr() if bits == 8 else None, self.buf[3].data_ptr(), 0, stream())

    def gradients(self, seed, scale=1.0):
        """New ones, times `scale`; padding zero."""
        gen = torch.Generator().manual_seed(seed)
        for i, unit in enumerate(self.c):
            used = sum(SHARDED) if self.calls == [-1] else sum(SHARDED[2 * i:2 * i + 2])
            for c in unit:
                c[:used] = (torch.randn(used, generator=gen) * 1e-2 * scale).to(torch.bfloat16).cuda()
        for o, n in zip(self.offs, REST):
            self.rest[o:o + n] = (torch.randn(n, generator=gen) * 1e-2 * scale).to(self.rest.dtype).cuda()

    def step(self, hyper, late=False, wait=True):
        contribs = [[c.data_ptr() for c in unit] for unit in self.c]
        if hyper.max_grad_norm > 0:
            for i, which in enumerate(self.calls):
                self.g.grad_norm(contribs[i], which)
        if not late:
            Z.zero_adamw_check(self.h, self.g.plan, stream())
        for i, which in enumerate(self.calls):
            self.g.step(contribs[i], which, hyper)
        if late:
            Z.zero_adamw_check(self.h, self.g.plan, stream())
        Z.zero_adamw_step_with(self.h, self.g.plan, hyper, stream())
        return self.g.finish(wait=wait)

    def state(self):
        """Everything that a step changes, as it is now."""
        out = [self.p, self.p16] + self.buf[:3]
        for r in range(self.n_d):
            out += [self.g.state_tensor(r, k) for k in ("master", "m", "v")]
            out += [self.g.shard16[r]] if self.g.stage == 3 else []
        out += [self.g.full16] if self.g.full16 is not None else []
        torch.cuda.synchronize()
        return [t.clone() for t in out]

    def flat(self, name):
        """The sharded master, m or v and the rest's, one float64 vector (ranks, then units, then tensors)."""
        parts = [self.g.logical(r, self.g.state_tensor(r, name)).double().cuda() for r in range(self.n_d)]
        if name == "master":
            parts += [self.p[o:o + n].double() for o, n in zip(self.offs, REST)]
        else:
            q = self.buf[0 if name == "m" else 1].view(torch.float32)
            at = 0
            for n in REST:
                parts.append(q[at:at + n].double())
                at += -(-n // Z.ZERO_ADAMW_BLOCK) * Z.ZERO_ADAMW_BLOCK
        return torch.cat(parts)

    def flat_gradient(self):
        parts = []
        for r in range(self.n_d):
            for u, _off, n, _base, _size in self.g.shard_slices(r):
                unit = self.c[u if self.calls != [-1] else 0]
                parts.append(torch.stack([c.double()[r * n:(r + 1) * n] for c in unit]).mean(0))
        return torch.cat(parts + [self.rest[o:o + n].double() for o, n in zip(self.offs, REST)])

    def close(self):
        torch.cuda.synchronize()
        Z.zero_adamw_destroy(self.h)
        self.g.close()


@pytest.mark.parametrize("stage", [2, 3])
@pytest.mark.parametrize("clip", [0.0, 0.3])
@pytest.mark.parametrize("scale", [1.0, 1024.0])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
def test_one_adamw_over_all_parameters(stage, clip, scale, grad):
    both = Both(stage, grad=grad)
    try:
        if scale != 1.0:
            both.g.set_scaler(Z.zero_scaler_t(scale, 2.0, 0.5, 1.0, 1000, 0))
        m = v = torch.zeros_like(both.flat("m"))
        for t in (1, 2, 3):
            both.gradients(t, scale)
            p, g = both.flat("master"), both.flat_gradient() / scale
            norm = math.sqrt(float((g * g).sum()))
            h = Z.hyper(max_grad_norm=clip * norm)
            if clip:
                g = g * min(1.0, h.max_grad_norm / (norm + 1e-6))
            res = both.step(h)
            assert res.t == t and not res.skipped
            if clip:
                assert abs(res.grad_norm - norm) <= 16 * U * norm
            m1, v1 = h.beta1 * m + (1 - h.beta1) * g, h.beta2 * v + (1 - h.beta2) * g * g
            dm = 12 * U * ((h.beta1 * m).abs() + ((1 - h.beta1) * g).abs()) + 2.0 ** -149
            dv = 24 * U * v1 + 2.0 ** -148
            bc1, bc2 = 1 - h.beta1 ** t, 1 - h.beta2 ** t
            d = (v1 / bc2).sqrt() + h.eps
            step = h.lr / bc1 * m1 / d
            want = p * (1 - h.lr * h.weight_decay) - step
            dd = torch.minimum(dv / (2 * v1.sqrt()).clamp(min=1e-300), dv.sqrt()) / math.sqrt(bc2)
            dp = 4 * U * p.abs() + 16 * U * step.abs() + h.lr / bc1 * (dm / d + m1.abs() / d * dd / (d - dd).clamp(min=h.eps))
            for name, w, bound in (("m", m1, dm), ("v", v1, dv), ("master", want, dp)):
                off = (both.flat(name) - w).abs()
                assert bool((off <= bound).all()), (name, t, float((off / bound).max()))
            m, v = both.flat("m"), both.flat("v")
    finally:
        both.close()


# a step that clips or is offloaded takes the check first
@pytest.mark.parametrize("offload,late,clip", [(False, False, 0.0), (False, False, 0.1), (False, True, 0.0), (True, False, 0.0),
                                               (True, False, 0.1)])
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("where", ["sharded", "rest"])
def test_a_step_is_left_out_whole(offload, bits, bad, where, late, clip):
    both, ref = Both(bits=bits, offload=offload), Both(bits=bits, offload=offload)
    h = Z.hyper(max_grad_norm=clip)
    try:
        for b in (both, ref):
            b.g.set_scaler(Z.zero_scaler_t(1.0, 2.0, 0.5, 0.125, 1000, 0))
            b.gradients(1)
            b.step(h, late)
        kept = both.state()
        both.gradients(2)
        if where == "sharded":
            both.c[1][1][3] = bad
        else:
            both.rest[both.offs[3] + 512] = bad
        res = both.step(h, late)
        assert res.skipped == 1 and res.t == 1 and res.scale == 0.5
        mine = Z.zero_adamw_read(both.h, stream())
        assert (mine.skipped, mine.t, mine.skipped_total, mine.finished) == (1, 1, 1, 2)
        assert all(torch.equal(a, b) for a, b in zip(kept, both.state()))
        # the next step is the one that a run without it makes
        both.g.set_scaler(Z.zero_scaler_t(1.0, 2.0, 0.5, 0.125, 1000, 0))
        for b in (both, ref):
            b.gradients(3)
            res = b.step(h, late)
            assert res.skipped == 0 and res.t == 2
        assert all(torch.equal(a, b) for a, b in zip(ref.state(), both.state()))
    finally:
        both.close()
        ref.close()


def test_without_clipping_and_scale_it_is_the_step_alone():
    both, alone = Both(bits=8), Both(bits=8)
    try:
        for t in (1, 2):
            for b in (both, alone):
                b.gradients(t)
            both.step(Z.hyper(), wait=False)
            Z.zero_adamw_step(alone.h, Z.hyper(), 1.0, stream())
            torch.cuda.synchronize()
            for a, b in zip([both.p, both.p16] + both.buf[:3], [alone.p, alone.p16] + alone.buf[:3]):
                assert torch.equal(a, b)
    finally:
        both.close()
        alone.close()


@pytest.mark.parametrize("clip", [0.0, 1.0])
def test_a_sum_of_squares_beyond_the_range_leaves_the_step_out(clip):
    """As zero_adamw_step's own norm pass does: the gradient is finite, its square is not."""
    both = Both()
    try:
        kept = both.state()
        both.gradients(1)
        both.rest[both.offs[1]] = 1e25
        res = both.step(Z.hyper(max_grad_norm=clip))
        assert res.skipped == 1 and res.t == 0 and Z.zero_adamw_read(both.h).skipped == 1
        kept2 = both.state()
        assert all(torch.equal(a, b) for a, b in zip(kept, kept2))
    finally:
        both.close()


def test_order():
    both = Both()
    plan, h, contribs = both.g.plan, Z.hyper(), [[c.data_ptr() for c in unit] for unit in both.c]

    def refused(status, f, *args):
        with pytest.raises(Z.ZeroError) as e:
            f(*args)
        assert e.value.status == status, str(e.value)

    try:
        both.gradients(1)
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, both.h, plan, h, stream())           # nothing open
        both.g.step(contribs[0], 0, h)
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, both.h, plan, h, stream())           # no check
        Z.zero_adamw_check(both.h, plan, stream())
        refused(Z.ZERO_ESTATE, Z.zero_adamw_check, both.h, plan, stream())                  # twice
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, both.h, plan, h, stream())           # a unit is missing
        both.g.step(contribs[1], 1, h)
        refused(Z.ZERO_EINVAL, Z.zero_adamw_step_with, both.h, plan, Z.hyper(max_grad_norm=1.0), stream())
        Z.zero_adamw_step_with(both.h, plan, h, stream())
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, both.h, plan, h, stream())           # twice
        assert both.g.finish().t == 1
        refused(Z.ZERO_ESTATE, Z.zero_adamw_step_with, both.h, plan, h, stream())
        # a clipping step takes the check before its first unit
        h = Z.hyper(max_grad_norm=1.0)
        for u in range(2):
            both.g.grad_norm(contribs[u], u)
        both.g.step(contribs[0], 0, h)
        refused(Z.ZERO_ESTATE, Z.zero_adamw_check, both.h, plan, stream())
        both.g.step(contribs[1], 1, h)
        assert both.g.finish().t == 2
    finally:
        both.close()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("where", ["matrices", "vectors"])
def test_a_network_is_left_whole_by_a_step_that_is_not_finite(bad, where):
    from zero_sharded_mixed_03_gb300.feed_forward import ShardedFeedForward
    model = ShardedFeedForward(2, 128, 256, 2, 64)
    try:
        gen = torch.Generator(device="cuda").manual_seed(0)

        def gradients():
            for r in range(2):
                x = torch.randn(64, 128, generator=gen, device="cuda").to(torch.bfloat16)
                model.forward(x)
                model.backward(r, x)

        def parts():
            torch.cuda.synchronize()
            return [t.clone() for t in [model.vectors, model.vectors16] + model.moments[:3]
                    + [model.group.state_tensor(r, k) for r in range(2) for k in ("master", "m", "v")]
                    + [model.group.shard16[r] for r in range(2)]]

        for h in (Z.hyper(lr=1e-3), Z.hyper(lr=1e-3, max_grad_norm=1.0)):
            gradients()
            model.step(h)
            before = parts()
            gradients()
            (model.contribs[1][0] if where == "matrices" else model.rank_vector_grads[1].view(-1))[5] = bad
            model.step(h)
            assert all(torch.equal(a, b) for a, b in zip(before, parts()))
            gradients()
            model.step(h)
            after = parts()
            assert all(bool(torch.isfinite(t.float()).all()) for t in after if t.dtype != torch.uint8)
            assert not torch.equal(after[0], before[0])
        assert model.group.step_state().t == Z.zero_adamw_read(model.opt).t == 4
    finally:
        torch.cuda.synchronize()
        model.close()
