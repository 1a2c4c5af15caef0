"""zero_adamw over more blocks than its grid has warps: each warp takes several, one after another.

The 8-bit moments' codes, scales and values, and the moments in 32 bits, are those of the rule
bit for bit: every product and sum of a moment is rounded by itself, and its code follows from the values alone.
The plain form of the rule is here in fp32 operations, one rounding each.
"""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z
from test_gpu_adamw import BLOCK, Opt, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()


def sizes_of(kind):
    if kind == "large":                    # 4.2M elements: 16,500 blocks of one kind
        return [3_000_000, 1_200_000 + 77]
    u = np.random.RandomState(5).random_sample(900)         # whole, inner and ragged blocks in turn
    return [int(n) for n in np.floor(2.0 ** (5 + 11 * u))] + [1, 0, 255, 256, 257, 511, 512, 513]


def power(e):
    return (e.to(torch.int32) << 23).view(torch.float32)


def top(x):
    return x.reshape(-1, BLOCK).abs().amax(1).view(torch.int32) >> 23


def encode_m(m):
    """e4m3 codes with the block's scale; values are on the format's grid after rounding to 8 bits."""
    e = (top(m) - 7).clamp(min=1)
    return (m.reshape(-1, BLOCK) * power(254 - e)[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1), e


def decode_m(codes, e):
    return (codes.view(torch.float8_e4m3fn).float().reshape(-1, BLOCK) * power(e)[:, None]).reshape(-1)


def encode_root(r):
    """Nearest of the 240 values of 4 exponent and 4 fraction bits, ties to the even code; none above 0 is 0."""
    e = top(r)
    y = r.reshape(-1, BLOCK).double() * torch.exp2(127.0 - e.double())[:, None]
    spacing = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -13))) - 4)
    q = torch.round(y / spacing) * spacing                   # torch.round: ties to even
    q = torch.where(y > 0, q.clamp(min=2.0 ** -17), q)
    field = torch.floor(torch.log2(q.clamp(min=2.0 ** -13))) + 14           # 14: [1, 2)
    code = torch.where(q >= 2.0 ** -13, field * 16 + (q * torch.exp2(14 - field) - 1) * 16, q * 2.0 ** 17)
    return code.to(torch.uint8).reshape(-1), e


def decode_root(codes, e):
    c = codes.double().reshape(-1, BLOCK)
    field = torch.floor(c / 16)
    y = torch.where(field > 0, torch.exp2(field - 14) * (1 + (c - 16 * field) / 16), c * 2.0 ** -17)
    return (y * torch.exp2(e.double() - 127)[:, None]).float().reshape(-1)


class Rule:
    """The step on padded fp32 vectors."""

    def __init__(self, opt):
        self.opt, n = opt, opt.info.state_elems
        place = []
        at = 0
        for size in opt.sizes:
            place.append(np.arange(at, at + size))
            at += -(-size // BLOCK) * BLOCK
        self.place = torch.from_numpy(np.concatenate(place)).cuda()
        self.m, self.root, self.v = (torch.zeros(n, device="cuda") for _ in range(3))
        self.from_ = torch.from_numpy(np.concatenate([o + np.arange(s) for o, s in zip(opt.offs, opt.sizes)])).cuda()

    def spread(self, buf):
        out = torch.zeros_like(self.m)
        out[self.place] = buf[self.from_].float()
        return out

    def step(self, h, t, coef=1.0):
        f = lambda x: float(np.float32(x))  # noqa: E731
        g, p = self.spread(self.opt.g) * f(coef), self.spread(self.opt.p)
        b1, c1, b2, c2 = (torch.full((), f(x), device="cuda") for x in (h.beta1, 1 - h.beta1, h.beta2, 1 - h.beta2))
        v = self.root * self.root if self.opt.bits == 8 else self.v
        m = torch.add(self.m * b1, g * c1)
        v = torch.add(v * b2, (g * g) * c2)
        root = v.sqrt()
        want = p.double() * (1 - h.lr * h.weight_decay) - h.lr / (1 - h.beta1 ** t) * m.double() / (
            v.double().sqrt() / math.sqrt(1 - h.beta2 ** t) + h.eps)
        step = (want - p.double()).abs()
        if self.opt.bits == 8:
            self.mc, self.me = encode_m(m)
            self.rc, self.re = encode_root(root)
            self.m, self.root = decode_m(self.mc, self.me), decode_root(self.rc, self.re)
        else:
            self.m, self.v = m, v
        # decay, step and parameter: at most 4 roundings of |p| and 16 of the step
        return want[self.place], (4 * U * p.double().abs() + 16 * U * step)[self.place] + 2.0 ** -149


def check_state(opt, rule):
    if opt.bits == 32:
        assert torch.equal(opt.m, rule.m) and torch.equal(opt.v, rule.v)
        return
    scales = opt.scales.view(-1, 2).int()
    assert torch.equal(scales[:, 0], rule.me.int()) and torch.equal(scales[:, 1], rule.re.int())
    off = opt.m != rule.mc                                 # the sign of a zero is not part of a value
    assert torch.equal(decode_m(opt.m, rule.me)[off], rule.m[off])
    assert torch.equal(opt.v, rule.rc)


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind", ["large", "ragged"])
@pytest.mark.parametrize("grad,p16", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16")])
@pytest.mark.parametrize("shift,align", [(0, 8), (1, 1)])
def test_codes_and_parameters(bits, kind, grad, p16, shift, align):
    opt = Opt(sizes_of(kind), bits, grad, p16, shift, align)
    assert opt.info.n_blocks > 8192 or kind == "ragged" and opt.info.n_blocks > 2 * 3648
    rule, h = Rule(opt), Z.hyper()
    try:
        gen = torch.Generator(device="cuda").manual_seed(3)
        for t in (1, 2, 3):
            size = torch.exp2(3 * torch.randn(opt.g.numel(), generator=gen, device="cuda"))
            opt.g.copy_((torch.randn(opt.g.numel(), generator=gen, device="cuda") * 1e-3 * size).to(opt.gt))
            before, before16 = opt.p.clone(), opt.p16.clone()
            want, bound = rule.step(h, t)
            opt.step(h)
            got = opt.p[rule.from_].double()
            assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
            check_state(opt, rule)
            assert torch.equal(opt.p16[rule.from_], opt.p[rule.from_].to(opt.p16.dtype))
            outside = torch.ones(opt.p.numel(), dtype=torch.bool, device="cuda")
            outside[rule.from_] = False
            assert torch.equal(opt.p[outside], before[outside]) and torch.equal(opt.p16[outside], before16[outside])
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind", ["large", "ragged"])
@pytest.mark.parametrize("grad", ["bf16", "fp32"])
@pytest.mark.parametrize("shift,align", [(0, 8), (1, 1)])
def test_clipped(bits, kind, grad, shift, align):
    """The norm over many blocks to a double's nearest fp32 coefficient, and the same codes behind it."""
    opt = Opt(sizes_of(kind), bits, grad, "bf16", shift, align)
    rule = Rule(opt)
    try:
        gen = torch.Generator(device="cuda").manual_seed(4)
        for t in (1, 2):
            opt.g.copy_((torch.randn(opt.g.numel(), generator=gen, device="cuda") * 1e-2).to(opt.gt))
            g = opt.g[rule.from_].float()
            norm = math.sqrt(float((g * g).double().sum()))
            h = Z.hyper(max_grad_norm=0.25 * norm)
            coef = np.float32(min(1.0, h.max_grad_norm / (norm + 1e-6)))
            want, bound = rule.step(h, t, coef)
            opt.step(h)
            res = Z.zero_adamw_read(opt.h, torch.cuda.current_stream().cuda_stream)
            # sums of fp32 squares: exact pairs of floats in each thread, doubles after them
            assert abs(res.grad_norm - norm) <= 2.0 ** -40 * norm
            near = np.float32(min(1.0, h.max_grad_norm / (res.grad_norm + 1e-6)))
            assert near == coef, "the case's coefficient lies between two floats: choose another seed"
            got = opt.p[rule.from_].double()
            assert bool(((got - want).abs() <= bound).all()), float(((got - want).abs() / bound).max())
            check_state(opt, rule)
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
def test_one_gradient_of_millions_that_is_not_finite(bits):
    opt = Opt(sizes_of("ragged"), bits, "bf16", "bf16", 1)
    try:
        opt.step(Z.hyper())
        kept = [b.clone() for b in (opt.p, opt.p16, opt.m, opt.v, opt.scales)]
        for at in (opt.offs[0], opt.offs[400] + 3, opt.offs[-1] + 512):
            old = opt.g[at].clone()
            opt.g[at] = math.nan
            opt.step(Z.hyper(report_grad_norm=True))
            assert all(torch.equal(a, b) for a, b in zip(kept, (opt.p, opt.p16, opt.m, opt.v, opt.scales)))
            opt.g[at] = old
        assert Z.zero_adamw_read(opt.h).skipped_total == 3
    finally:
        opt.close()
