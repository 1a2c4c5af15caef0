"""zero_adamw (one AdamW step over many tensors, moments in 8 or 32 bits) against float64.

Tolerances.  u = 2^-24 is one fp32 rounding.  A new moment is a sum of two products with constants
rounded once: 4 roundings of magnitudes |b1 m| and |(1-b1) g| (g itself two more where it is
unscaled and clipped), so |dm| <= 8 u (|b1 m| + |(1-b1) g|), and twice g's part for g^2.  The
parameter adds the decay (3 roundings) and the step lr/bc1 m/d: the errors of m and v relative to
their magnitudes (half of v's in its root), and 8 more roundings.  An 8-bit moment is half a
spacing of its format from the fp32 one.
"""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BLOCK = Z.ZERO_ADAMW_BLOCK
GRADS = {"bf16": (torch.bfloat16, Z.ZERO_BF16), "fp16": (torch.float16, Z.ZERO_FP16),
         "fp32": (torch.float32, Z.ZERO_FP32)}
SIZES = [1, 7, 0, 255, 256, 257, 1000, 8, 4099, 65536 + 17]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()


class Opt:
    """Tensors carved from flat buffers with `gap` elements between them, bound to a handle."""

    def __init__(self, sizes, bits, grad="bf16", p16="bf16", shift=0, align=1, t=0, guard=64, seed=0):
        self.sizes, self.bits = list(sizes), bits
        self.gt, gk = GRADS[grad]
        self.h = Z.zero_adamw_create(self.sizes, bits, Z.ZERO_BF16 if p16 != "fp16" else Z.ZERO_FP16, gk)
        self.info = Z.zero_adamw_info(self.h)
        self.offs, at = [], guard + shift
        for n in self.sizes:
            at = -(-at // align) * align if align > 1 else at
            self.offs.append(at)
            at += n
        total = at + guard
        gen = torch.Generator().manual_seed(seed)
        self.p = torch.randn(total, generator=gen).mul(0.02).cuda()
        self.g = torch.randn(total, generator=gen).mul(1e-2).to(self.gt).cuda()
        self.p16 = None if p16 is None else torch.full((total,), 7.0, dtype=GRADS[p16][0], device="cuda")
        n = self.info.state_elems
        kind = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = torch.zeros(n, dtype=kind, device="cuda"), torch.zeros(n, dtype=kind, device="cuda")
        self.scales = torch.zeros(max(2, self.info.scale_bytes), dtype=torch.uint8, device="cuda")
        self.ws = torch.full((self.info.workspace_bytes,), 0xAB, dtype=torch.uint8, device="cuda")
        self.bind(t)

    def ptrs(self, buf):
        return [buf.data_ptr() + o * buf.element_size() for o in self.offs]

    def bind(self, t):
        Z.zero_adamw_bind(self.h, self.ptrs(self.p), self.ptrs(self.p16) if self.p16 is not None else None,
                          self.ptrs(self.g), self.m.data_ptr(), self.v.data_ptr(),
                          self.scales.data_ptr() if self.bits == 8 else None, self.ws.data_ptr(), t,
                          torch.cuda.current_stream().cuda_stream)

    def step(self, hyper, loss_scale=1.0):
        Z.zero_adamw_step(self.h, hyper, loss_scale, torch.cuda.current_stream().cuda_stream)

    def tensors(self, buf):
        a = buf.double().cpu().numpy()
        return np.concatenate([a[o:o + n] for o, n in zip(self.offs, self.sizes)] or [np.zeros(0)])

    def moments(self):
        """(m, root of v) over the tensors, float64, as stored."""
        if self.bits == 32:
            m, r = self.m.double(), self.v.double().sqrt()
        else:
            out = [torch.empty(self.info.state_elems, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            Z.zero_adamw_export(self.h, out[0].data_ptr(), out[1].data_ptr(), torch.cuda.current_stream().cuda_stream)
            m, r = out[0].double(), out[1].double()
        return self.unpad(m.cpu().numpy()), self.unpad(r.cpu().numpy())

    def unpad(self, a):
        out, b = [], 0
        for n in self.sizes:
            out.append(a[b:b + n])
            pad = a[b + n:b + -(-n // BLOCK) * BLOCK]
            assert not np.any(pad), "the moments' padding is not zero"
            b += -(-n // BLOCK) * BLOCK
        return np.concatenate(out) if out else np.zeros(0)

    def block_of(self):
        out, b = [], 0
        for n in self.sizes:
            out.append(b + np.arange(n) // BLOCK)
            b += -(-n // BLOCK)
        return np.concatenate(out).astype(np.int64)

    def close(self):
        torch.cuda.synchronize()
        Z.zero_adamw_destroy(self.h)


def reference(p, g, m, root, t, h, loss_scale=1.0, max_norm=0.0):
    """One step in float64: (p, m, v, bounds of p and m and v)."""
    g = g / loss_scale
    if max_norm > 0:
        g = g * min(1.0, max_norm / (math.sqrt(float((g * g).sum())) + 1e-6))
    b1, b2 = h.beta1, h.beta2
    v = root ** 2
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    dm = 8 * U * (abs(b1 * m) + abs((1 - b1) * g)) + 2.0 ** -149
    dv = 12 * U * v1 + 2.0 ** -148
    bc1, bc2 = 1 - b1 ** t, 1 - b2 ** t
    d = np.sqrt(v1 / bc2) + h.eps
    step = h.lr / bc1 * m1 / d
    p1 = p * (1 - h.lr * h.weight_decay) - step
    # |d sqrt(v)| <= min(dv / (2 sqrt v), sqrt dv)
    dd = np.minimum(dv / np.maximum(2 * np.sqrt(v1), 1e-300), np.sqrt(dv)) / math.sqrt(bc2)
    dp = 4 * U * abs(p) + 8 * U * abs(step) + h.lr / bc1 * (dm / d + abs(m1) / d * dd / np.maximum(d - dd, h.eps))
    return p1, m1, v1, dp, dm, dv


def check(opt, h, t, loss_scale=1.0, max_norm=0.0):
    p0, g0 = opt.tensors(opt.p), opt.tensors(opt.g)
    m0, r0 = opt.moments()
    before = opt.p.clone(), opt.p16.clone() if opt.p16 is not None else None
    opt.step(h, loss_scale)
    p1, m1, v1, dp, dm, dv = reference(p0, g0, m0, r0, t, h, loss_scale, max_norm)
    got = opt.tensors(opt.p)
    assert np.all(abs(got - p1) <= dp), float((abs(got - p1) / dp).max())
    gm, gr = opt.moments()
    r1 = np.sqrt(v1)
    dr = np.minimum(dv / np.maximum(2 * r1, 1e-300), np.sqrt(dv)) + U * r1
    if opt.bits == 8:
        e = opt.scales.cpu().numpy().reshape(-1, 2)[opt.block_of()].astype(np.float64)
        # half a spacing of e4m3 (subnormals below 2^-6), of the 4 + 4 bit root (below 2^-13)
        x = abs(m1) / 2.0 ** (e[:, 0] - 127)
        assert np.all(x <= 448)
        dm = dm + 0.5 * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(x, 1e-300))), -6) - 3 + e[:, 0] - 127) * (1 + 1e-6)
        y = r1 / 2.0 ** np.where(e[:, 1] > 0, e[:, 1] - 127, 0)
        assert np.all(y <= 2 * (1 + 1e-6))
        half = 0.5 * 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(y, 1e-300))), -13) - 4 + e[:, 1] - 127)
        dr = dr + np.where(r1 > 0, half * (1 + 1e-6), 0)
        low = (r1 > 0) & (y < 2.0 ** -17)
        dr = dr + np.where(low, 2.0 ** (e[:, 1] - 127 - 17), 0)
        assert np.all(gr[r1 > 2 * np.sqrt(2.0 ** -148)] > 0)
        # scales follow the block's largest value (a power of two apart only at a boundary)
        top = np.zeros(opt.info.n_blocks)
        np.maximum.at(top, opt.block_of(), abs(m1))
        want = np.maximum(np.floor(np.log2(np.maximum(top, 2.0 ** -126))) + 127 - 7, 1)
        have = opt.scales.cpu().numpy().reshape(-1, 2)[:, 0]
        near = abs(np.log2(np.maximum(top, 2.0 ** -126)) - np.rint(np.log2(np.maximum(top, 2.0 ** -126)))) < 1e-5
        assert np.all((have == want) | (near & (abs(have - want) <= 1)))
    assert np.all(abs(gm - m1) <= dm), float((abs(gm - m1) / dm).max())
    assert np.all(abs(gr - r1) <= dr + 1e-45), float((abs(gr - r1) / (dr + 1e-45)).max())
    # the 16-bit copy is the parameter's rounding; nothing between the tensors was touched
    inside = torch.zeros(opt.p.numel(), dtype=torch.bool)
    for o, n in zip(opt.offs, opt.sizes):
        inside[o:o + n] = True
    inside = inside.cuda()
    assert torch.equal(opt.p[~inside], before[0][~inside])
    if opt.p16 is not None:
        assert torch.equal(opt.p16[inside], opt.p[inside].to(opt.p16.dtype))
        assert torch.equal(opt.p16[~inside], before[1][~inside])


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad,p16", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16"), ("fp32", None)])
@pytest.mark.parametrize("shift,align", [(0, 1), (1, 1), (0, 8), (4, 8)])
def test_steps(bits, grad, p16, shift, align):
    opt = Opt(SIZES, bits, grad, p16, shift, align)
    try:
        for t in (1, 2, 3, 4):
            opt.g.copy_((torch.randn(opt.g.numel(), generator=torch.Generator().manual_seed(t)) * 1e-2).to(opt.gt))
            check(opt, Z.hyper(), t)
        res = Z.zero_adamw_read(opt.h, torch.cuda.current_stream().cuda_stream)
        assert (res.t, res.finished, res.skipped, res.grad_norm) == (4, 4, 0, -1.0)
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("spread", [1e-30, 1e-8, 1.0, 1e6, 1e15])
def test_ranges(bits, spread):
    """Blocks whose values span 18 binades of a common scale, exact zeros among them."""
    opt = Opt([700, 256, 33], bits, "fp32", None)
    try:
        for t in (1, 2, 3):
            gen = torch.Generator().manual_seed(100 + t)
            n = opt.g.numel()
            g = torch.randn(n, generator=gen) * torch.exp2(-18 * torch.rand(n, generator=gen)) * spread
            opt.g.copy_(torch.where(torch.rand(n, generator=gen) < 0.1, torch.zeros(n), g))
            check(opt, Z.hyper(eps=1e-8 * spread), t)
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
def test_zero_gradients_only_decay(bits):
    opt = Opt([300, 5], bits)
    try:
        opt.g.zero_()
        p = opt.tensors(opt.p)
        opt.step(Z.hyper(lr=0.1, weight_decay=0.5))
        assert np.all(abs(opt.tensors(opt.p) - p * 0.95) <= 3 * U * abs(p))
        m, r = opt.moments()
        assert not m.any() and not r.any()
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("grad", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift", [0, 3])
def test_clipping_and_loss_scale(bits, grad, shift):
    opt = Opt(SIZES, bits, grad, "bf16", shift)
    try:
        norm = math.sqrt(float((opt.tensors(opt.g) / 64) @ (opt.tensors(opt.g) / 64)))
        for t, max_norm in ((1, 0.5 * norm), (2, 2.0 * norm)):
            check(opt, Z.hyper(max_grad_norm=max_norm), t, 64.0, max_norm)
            res = Z.zero_adamw_read(opt.h, torch.cuda.current_stream().cuda_stream)
            assert abs(res.grad_norm - norm) <= 2 * U * norm and res.t == t
    finally:
        opt.close()


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_step_that_is_not_finite_is_skipped(bits, bad):
    opt = Opt(SIZES, bits, "fp16", "fp16")
    try:
        check(opt, Z.hyper(), 1)
        kept = [b.clone() for b in (opt.p, opt.p16, opt.m, opt.v, opt.scales)]
        at = opt.offs[-1] + 1000
        old = opt.g[at].clone()
        opt.g[at] = bad
        opt.step(Z.hyper(report_grad_norm=True))
        assert all(torch.equal(a, b) for a, b in zip(kept, (opt.p, opt.p16, opt.m, opt.v, opt.scales)))
        res = Z.zero_adamw_read(opt.h, torch.cuda.current_stream().cuda_stream)
        assert (res.t, res.finished, res.skipped, res.skipped_total) == (1, 2, 1, 1) and math.isnan(res.grad_norm)
        opt.g[at] = old
        check(opt, Z.hyper(report_grad_norm=True), 2)
    finally:
        opt.close()


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_unchecked_gradient_spoils_its_own_element_only(bad):
    opt = Opt([600], 8, "fp32", None)
    try:
        opt.g[opt.offs[0] + 300] = bad
        opt.step(Z.hyper())
        opt.g[opt.offs[0] + 300] = 0.0
        opt.step(Z.hyper())
        p = opt.tensors(opt.p)
        m, r = opt.moments()
        for a in (p, m, r):
            assert not np.isfinite(a[300]) and np.all(np.isfinite(np.delete(a, 300)))
        assert np.all(np.delete(r, 300) > 0)
    finally:
        opt.close()


def test_eight_bit_moments_train_like_32_bit_ones():
    """A quadratic: both end at the same loss, within a factor that half a spacing allows."""
    losses = {}
    for bits in (8, 32):
        opt = Opt([4096], bits, "fp32", None, align=8)
        try:
            target = torch.randn(opt.p.numel(), generator=torch.Generator().manual_seed(5)).cuda() * 0.1
            for _ in range(300):
                torch.sub(opt.p, target, out=opt.g)
                opt.step(Z.hyper(lr=2e-3, weight_decay=0.0))
            sl = slice(opt.offs[0], opt.offs[0] + 4096)
            losses[bits] = float((opt.p[sl] - target[sl]).square().mean())
        finally:
            opt.close()
    start = 0.1 ** 2
    assert losses[32] < 1e-3 * start and losses[8] < 1e-3 * start, losses


def test_rebind_keeps_the_count_and_other_streams_and_graphs_work():
    opt = Opt(SIZES, 8, "bf16", "bf16")
    ref = Opt(SIZES, 8, "bf16", "bf16")
    side = torch.cuda.Stream()
    try:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            opt.step(Z.hyper())
            opt.g = opt.g.clone()
            opt.bind(-1)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            opt.step(Z.hyper(max_grad_norm=0.1))
        graph.replay()
        graph.replay()
        ref.step(Z.hyper())
        for _ in range(2):
            ref.step(Z.hyper(max_grad_norm=0.1))
        torch.cuda.synchronize()
        assert Z.zero_adamw_read(opt.h).t == Z.zero_adamw_read(ref.h).t == 3
        for a, b in ((opt.p, ref.p), (opt.p16, ref.p16), (opt.m, ref.m), (opt.v, ref.v), (opt.scales, ref.scales)):
            assert torch.equal(a, b)
    finally:
        opt.close()
        ref.close()


def test_resumed_at_a_late_step():
    opt = Opt([1000], 32, "fp32", None, t=99_999)
    try:
        check(opt, Z.hyper(), 100_000)
        assert Z.zero_adamw_read(opt.h).t == 100_000
    finally:
        opt.close()


def test_no_tensors_and_empty_tensors():
    for sizes in ([], [0, 0]):
        opt = Opt(sizes, 8)
        try:
            opt.step(Z.hyper(max_grad_norm=1.0))
            assert Z.zero_adamw_read(opt.h).t == 1
        finally:
            opt.close()
