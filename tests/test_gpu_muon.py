"""zero_muon against float64.

Tolerances.  The momentum: the contributions' sum has n_contribs fp32 roundings, the mean, the product and the sum
three more, 2^-24 each, of the terms' magnitudes.  The orthogonalised X: what the iteration makes of roundings cannot
be bounded closely by norms (each step multiplies an error by up to 3.9), so the float64 iteration is run with every
operand that the kernels round to fp16 moved by half a step, 2^-11 of its value, with random signs; the tolerance is
twice the largest of the 2-norms by which eight such runs miss the unmoved one, and 2^-13 of the result for what fp32
sums add.  Half a step is the most that a rounding moves a value, its root mean square 0.4 of that.  Matrices whose
entries are powers of two, one at most in a row and a column, with dyadic coefficients, are exact.  Parameters: the
update and the decay are two fused operations, 2^-24 each of the terms.
"""
import math

import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z
from zero_sharded_mixed_03_gb300.emulate import EmulatedGroup

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ABC = (3.4445, -4.7750, 2.0315)
KINDS = {"bf16": (torch.bfloat16, Z.ZERO_BF16, 2.0 ** -8), "fp16": (torch.float16, Z.ZERO_FP16, 2.0 ** -11)}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def stream():
    return torch.cuda.current_stream().cuda_stream


class Muon:
    """Matrices in storage of their own, `shift` elements in, with guards around them."""

    def __init__(self, shapes, n_d=1, dtype="bf16", shift=0, params=True, updates=True, copies=True, t=0):
        self.t16, kind, self.u16 = KINDS[dtype]
        self.shapes, self.n_d, n = shapes, n_d, len(shapes)
        self.h = Z.zero_muon_create([r for r, _ in shapes], [c for _, c in shapes], n_d, kind)
        info = Z.zero_muon_info(self.h)
        new = lambda t: [self.guarded(r, c, t, shift) for r, c in shapes]  # noqa: E731
        self.p, self.p16, self.x = new(torch.float32), new(self.t16), new(self.t16)
        self.g = [new(self.t16) for _ in range(n_d)]
        self.halves = [torch.zeros(max(info.state_elems, 4), device="cuda") for _ in range(2)]
        self.at, at = [], 0
        for r, c in shapes:
            self.at.append(at)
            at += -(-r * c // 256) * 256
        self.ws = torch.full((info.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
        self.ptrs = [[v.data_ptr() if on and v.numel() else None for v in ts] for on, ts in
                     ((params, self.p), (params and copies, self.p16), (updates, self.x))]
        self.bind(t)

    def bind(self, t):
        Z.zero_muon_bind(self.h, *self.ptrs, [v.data_ptr() for g in self.g for v in g],
                         [v.data_ptr() for v in self.halves], self.ws.data_ptr(), t, stream())

    @staticmethod
    def guarded(r, c, t, shift):
        buf = torch.full((shift + r * c + 16,), 7.0, dtype=t, device="cuda")
        return buf[shift:shift + r * c].view(r, c)

    def guards_stand(self):
        for ts in (self.p, self.p16, self.x, *self.g):
            for v in ts:
                whole = torch.as_strided(v, (v.untyped_storage().nbytes() // v.element_size(),), (1,), 0)
                assert bool((whole[:v.storage_offset()] == 7).all()) and bool((whole[v.storage_offset() + v.numel():] == 7).all())

    def m(self, half, i):
        r, c = self.shapes[i]
        return self.halves[half][self.at[i]:self.at[i] + r * c].view(r, c)

    def fill(self, seed, scale=1e-3):
        gen = torch.Generator().manual_seed(seed)
        for i, (r, c) in enumerate(self.shapes):
            self.p[i].copy_(torch.randn(r, c, generator=gen) * 0.02)
            self.m(0, i).copy_(torch.randn(r, c, generator=gen) * scale)
            for k in range(self.n_d):
                self.g[k][i].copy_((torch.randn(r, c, generator=gen) * scale).to(self.t16))
        return self

    def step(self, hyper, loss_scale=1.0):
        Z.zero_muon_step(self.h, hyper, loss_scale, stream())
        return Z.zero_muon_read(self.h, stream())

    def close(self):
        torch.cuda.synchronize()
        Z.zero_muon_destroy(self.h)


def iterate(u, eps, abc, move=None, pair=False):
    """The definition in float64; move(x): x with every entry a half step of fp16 off, at the places where the kernels
    round (pair: the first two iterations made at once, as they are where every smaller side is at least 128)."""
    off = move or (lambda v: v)
    x = u / (torch.linalg.matrix_norm(u) + eps)
    wide = x.shape[0] <= x.shape[1]
    gram = lambda h: off(h @ h.t() if wide else h.t() @ h)  # noqa: E731
    times = lambda p, h: p @ h if wide else h @ p  # noqa: E731
    eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
    h = off(x)                              # the first of the two numbers that X is kept as
    first = 0
    if pair and len(abc) > 1:
        (a, b, c), (a2, b2, c2) = abc[:2]
        g = gram(h)
        r = off(b * g + c * (g @ g))
        w = off(r @ g)
        g = off(a * a * g + 2 * a * w + r @ w)
        s = off(b2 * g + c2 * (g @ g))
        h = off(times(off(a2 * r + a * s + s @ r), h) + a * a2 * x)
        first = 2
    for k, (a, b, c) in enumerate(abc[first:], first):
        g = gram(h)
        poly = b * g + c * (g @ g)
        if k < 2 and not pair:
            x = times(off(poly), h) + a * x
        else:
            x = times(off(poly + a * eye), h)
        h = off(x)
        if k >= 1 or pair:
            x = h
    return h if move else x


def tolerance(u, eps, abc, want, pair):
    gen = torch.Generator(device="cuda").manual_seed(1)

    def move(v):
        sign = torch.randint(0, 2, v.shape, generator=gen, device="cuda", dtype=torch.float64) * 2 - 1
        if v.shape[0] == v.shape[1]:
            sign = torch.triu(sign) + torch.triu(sign, 1).t()
        return v * (1 + 2.0 ** -11 * sign)

    worst = max(float((iterate(u, eps, abc, move, pair) - want).norm()) for _ in range(8))
    return 2 * worst + 2.0 ** -13 * float(want.norm()) + 1e-30


def expected(mu, case, i, half, hyper, loss_scale=1.0):
    """g, m', u of matrix i in float64, and the bound of m''s error."""
    g = sum(mu.g[k][i].double() for k in range(mu.n_d)) / (mu.n_d * loss_scale)
    mag = sum(mu.g[k][i].double().abs() for k in range(mu.n_d)) / (mu.n_d * loss_scale)
    old, b = mu.m(half, i).double(), hyper.momentum
    m = b * old + (1 - b) * g
    u = b * m + (1 - b) * g if hyper.flags & Z.ZERO_MUON_NESTEROV else m
    return g, m, u, (mu.n_d + 5) * U * ((1 - b) * mag + b * old.abs()) + 2.0 ** -149


def coefficients(hyper):
    return [tuple(hyper.coefficients[k]) for k in range(hyper.steps)]


def check(mu, hyper, half=0, loss_scale=1.0):
    """One step from the given half, X by way of parameters that are 0 (lr 1, no decay)."""
    want = [expected(mu, None, i, half, hyper, loss_scale) for i in range(len(mu.shapes))]
    before = [p.clone() for p in mu.p]
    res = mu.step(hyper, loss_scale)
    assert res.skipped == 0 and res.current == half ^ 1
    mu.guards_stand()
    for i, (r, c) in enumerate(mu.shapes):
        if r * c == 0:
            continue
        _g, m, u, err = want[i]
        assert bool(((mu.m(half ^ 1, i).double() - m).abs() <= err).all())
        x = iterate(u, hyper.eps, coefficients(hyper))
        tol = tolerance(u, hyper.eps, coefficients(hyper), x, min(min(s) for s in mu.shapes if min(s)) >= 128)
        if mu.ptrs[2][i]:
            got = mu.x[i].double()
            off = float((got - x).norm())
            assert off <= tol + mu.u16 * float(x.norm()) + 2.0 ** -25 * math.sqrt(r * c), (r, c, off, tol)
        if mu.ptrs[0][i]:
            s = {0: 1.0, 1: math.sqrt(max(1.0, r / c)), 2: 0.2 * math.sqrt(max(r, c))}[hyper.scale] * hyper.lr
            p = before[i].double() * (1 - hyper.lr * hyper.weight_decay) - s * x
            off = float((mu.p[i].double() - p).norm())
            assert off <= s * tol + 4 * U * float(p.norm() + before[i].norm() + s * x.norm()), (r, c, off, s * tol)
            if mu.ptrs[1][i]:
                assert torch.equal(mu.p16[i], mu.p[i].to(mu.t16))


SHAPES = [(1, 1), (1, 50), (50, 1), (5, 3), (16, 16), (24, 198), (130, 70), (128, 128), (257, 129), (300, 1000),
          (1000, 301), (520, 520)]


@pytest.mark.parametrize("r,c", SHAPES)
def test_against_float64(r, c):
    for dtype, n_d, nesterov, scale in (("bf16", 1, True, 2), ("fp16", 3, False, 1)):
        mu = Muon([(r, c)], n_d, dtype).fill(r + c)
        check(mu, Z.muon_hyper(lr=0.1, weight_decay=0.1, nesterov=nesterov, scale=scale))
        mu.p[0].zero_()
        check(mu, Z.muon_hyper(lr=1.0, weight_decay=0.0, nesterov=nesterov, scale=0), half=1)
        mu.close()


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 8])
def test_steps_and_coefficients(steps):
    abc = [ABC if k % 2 == 0 else (1.875, -1.25, 0.375) for k in range(steps)]
    mu = Muon([(200, 96), (96, 200)]).fill(steps)
    check(mu, Z.muon_hyper(steps=steps, coefficients=abc, momentum=0.0))
    mu.close()


def test_many_matrices():
    shapes = [(64, 200), (0, 5), (300, 40), (1, 9), (5, 0), (129, 129), (7, 1000), (640, 384), (384, 640)]
    for shift, dtype in ((0, "bf16"), (1, "bf16"), (8, "fp16"), (3, "fp16")):
        mu = Muon(shapes, 2, dtype, shift=shift).fill(shift)
        check(mu, Z.muon_hyper(lr=0.01))
        check(mu, Z.muon_hyper(lr=0.01), half=1)
        mu.close()


@pytest.mark.parametrize("sizes", [(2048, 700), (700, 2304), (1536, 1536)])
def test_tiles_of_256(sizes):
    mu = Muon([sizes] * 5, 5, "bf16").fill(3)
    check(mu, Z.muon_hyper())
    mu.close()


def test_without_parameters_or_updates():
    for params, updates, copies in ((True, False, True), (False, True, True), (True, True, False), (True, False, False)):
        mu = Muon([(96, 130), (130, 96)], 1, "bf16", params=params, updates=updates, copies=copies).fill(5)
        kept = [[v.clone() for v in ts] for ts in (mu.p, mu.p16, mu.x)]
        check(mu, Z.muon_hyper())
        for ts, old, bound in zip((mu.p, mu.p16, mu.x), kept, mu.ptrs):
            for v, o, ptr in zip(ts, old, bound):
                assert ptr or torch.equal(v, o)
        mu.close()


def partial_permutation(r, c, k, gen):
    """4^k entries +-2^3, one at most in a row and a column: norm 2^(k + 3)."""
    n = 4 ** k
    rows, cols = torch.randperm(r, generator=gen)[:n], torch.randperm(c, generator=gen)[:n]
    v = torch.zeros(r, c)
    v[rows, cols] = 8.0 * (torch.randint(0, 2, (n,), generator=gen) * 2 - 1)
    return v


@pytest.mark.parametrize("r,c,k", [(1, 1, 0), (5, 9, 1), (70, 64, 3), (64, 333, 2), (300, 257, 4), (512, 1100, 4),
                                   (1100, 512, 4), (1500, 1300, 5), (2050, 2050, 5)])
def test_exact(r, c, k):
    gen = torch.Generator().manual_seed(r)
    v = partial_permutation(r, c, k, gen)
    for n_d in (1, 4):
        mu = Muon([(r, c)], n_d, "bf16")
        for g in mu.g:
            g[0].copy_(v)
        # singular values 2^-k: x -> x (1.5 - 0.5 x^2), then (two steps where k < 2) x (1 + 0.25 x^2): from 1/2 11/16 and
        # 11/16 (1 + 121/1024), the polynomials' parts of at most 7 bits
        abc = [(1.5, -0.5, 0.0), (1.0, 0.25, 0.0)]
        hyper = Z.muon_hyper(lr=1.0, weight_decay=0.0, momentum=0.0, eps=1e-12, steps=1 if k > 1 else 2, coefficients=abc, scale=0)
        mu.p[0].zero_()
        mu.step(hyper)
        x = v.double().cuda() * 2.0 ** -(k + 3)
        for a, b, d in abc[:hyper.steps]:
            x = x * (a + b * x ** 2 + d * x ** 4)
        assert torch.equal(mu.p[0].double(), -x), float((mu.p[0].double() + x).abs().max())
        assert torch.equal(mu.x[0], x.float().to(torch.bfloat16))
        mu.guards_stand()
        mu.close()


@pytest.mark.parametrize("r,c", [(128, 128), (300, 257), (257, 1100), (2050, 2050)])
def test_exact_two_at_once(r, c):
    v = partial_permutation(r, c, 1, torch.Generator().manual_seed(r))
    mu = Muon([(r, c)], 1, "bf16")
    mu.g[0][0].copy_(v)
    mu.p[0].zero_()
    # singular values 1/2: G 1/4, R1 1/8, W 1/32, the second G 81/256 and R 81/512, Q 1241/4096
    mu.step(Z.muon_hyper(lr=1.0, weight_decay=0.0, momentum=0.0, eps=1e-12, steps=2, coefficients=(1.0, 0.5, 0.0), scale=0))
    x = v.double().cuda() / 16 * (5337 / 4096)
    assert torch.equal(mu.p[0].double(), -x)
    mu.close()


def test_zero_gradients_and_small_ones():
    mu = Muon([(40, 70), (40, 70)], 2, "fp16").fill(1)
    for g in mu.g:
        g[0].zero_()
        g[1].mul_(2.0 ** -6)
    for half in mu.halves:
        half.zero_()
    before = mu.p[0].clone()
    mu.step(Z.muon_hyper(weight_decay=0.0))
    assert torch.equal(mu.p[0], before) and not bool(mu.x[0].any())
    assert bool(torch.isfinite(mu.p[1]).all()) and bool(mu.x[1].any())
    mu.close()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), 3e38])
def test_a_step_that_is_not_finite_is_left_out(bad):
    mu = Muon([(40, 70), (90, 33)], 3, "bf16").fill(2)
    hyper = Z.muon_hyper()
    mu.step(hyper)
    good = mu.g[2][1][89, 32].clone()
    mu.g[2][1][89, 32] = bad
    kept = [v.clone() for ts in (mu.p, mu.p16, mu.x) for v in ts] + [mu.halves[1].clone()]
    for k in range(2):
        res = mu.step(hyper)
        assert (res.skipped, res.t, res.skipped_total, res.finished, res.current) == (1, 1, k + 1, k + 2, 1)
        now = [v for ts in (mu.p, mu.p16, mu.x) for v in ts] + [mu.halves[1]]
        assert all(torch.equal(a, b) for a, b in zip(kept, now))
    mu.g[2][1][89, 32] = good
    check(mu, hyper, half=1)
    assert Z.zero_muon_read(mu.h, stream()).t == 2
    mu.close()


def test_loss_scale():
    mu = Muon([(64, 96)], 2, "fp16").fill(4)
    for g in mu.g:
        g[0].mul_(1024.0)
    check(mu, Z.muon_hyper(), loss_scale=1024.0)
    mu.close()


def test_rebind_keeps_the_state():
    one, two = (Muon([(64, 96), (33, 20)], 1).fill(6) for _ in range(2))
    hyper = Z.muon_hyper(lr=0.01)
    for k in range(3):
        one.step(hyper)
        if k == 1:
            two.p = [v.clone() for v in two.p]
            two.ptrs[0] = [v.data_ptr() for v in two.p]
            two.bind(-1)
        two.step(hyper)
    assert all(torch.equal(a, b) for a, b in zip(one.p + one.halves, two.p + two.halves))
    assert Z.zero_muon_read(two.h, stream()).t == 3
    one.close()
    two.close()


def test_streams_graphs_and_repeats():
    shapes = [(300, 700), (700, 300), (65, 129)]
    hyper = Z.muon_hyper(lr=0.01)
    first, second, third = (Muon(shapes, 3, "bf16").fill(7) for _ in range(3))
    for _ in range(3):
        first.step(hyper)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            Z.zero_muon_step(second.h, hyper, 1.0, side.cuda_stream)
    side.synchronize()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_muon_step(third.h, hyper, 1.0, stream())
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for other in (second, third):
        assert all(torch.equal(a, b) for a, b in zip(first.p + first.p16 + first.x + first.halves,
                                                     other.p + other.p16 + other.x + other.halves))
    for mu in (first, second, third):
        mu.close()


def test_more_matrices_and_contributions():
    """More matrices than a block keeps marks of, and the most contributions."""
    for shapes, n_d in (([(40 + i % 7, 90 - i % 11) for i in range(70)], 2), ([(150, 130 + i) for i in range(66)], 1),
                        ([(33, 47), (130, 256)], 128)):
        mu = Muon(shapes, n_d).fill(n_d)
        check(mu, Z.muon_hyper())
        mu.close()


def test_calls_at_once():
    """Two optimizers and a linear layer's products on three streams."""
    shapes = [(700, 900), (260, 1300)]
    hyper = Z.muon_hyper(lr=0.01)
    alone, first, second = (Muon(shapes, 2, "bf16").fill(11) for _ in range(3))
    for _ in range(4):
        alone.step(hyper)
    x, w, y = (torch.randn(1024, 1024, device="cuda").bfloat16() for _ in range(3))
    args = Z.zero_linear_t(rows=1024, in_features=1024, out_features=1024, dtype16=Z.ZERO_BF16,
                           layout=Z.ZERO_WEIGHT_OUT_IN, x=x.data_ptr(), w=w.data_ptr(), y=y.data_ptr())
    n = Z.zero_linear_workspace(args)
    ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        Z.zero_muon_step(first.h, hyper, 1.0, streams[0].cuda_stream)
        Z.zero_linear(args, ws.data_ptr(), n, streams[2].cuda_stream)
        Z.zero_muon_step(second.h, hyper, 1.0, streams[1].cuda_stream)
    torch.cuda.synchronize()
    for other in (first, second):
        assert all(torch.equal(a, b) for a, b in zip(alone.p + alone.halves, other.p + other.halves))
    Z.zero_operators_check(stream())
    for mu in (alone, first, second):
        mu.close()


def test_no_matrices():
    mu = Muon([(0, 4)])
    assert mu.step(Z.muon_hyper()).t == 1
    mu.close()


def test_far_offsets():
    """A matrix of 2^32 elements and one behind it: entries in the far corners, exact."""
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("needs 120 GB")
    shapes, t16 = [(1024, 1 << 22), (70, 64)], torch.bfloat16
    h = Z.zero_muon_create([r for r, _ in shapes], [c for _, c in shapes], 1, Z.ZERO_BF16)
    info = Z.zero_muon_info(h)
    g = [torch.zeros(s, dtype=t16, device="cuda") for s in shapes]
    x = [torch.full(s, 3.0, dtype=t16, device="cuda") for s in shapes]
    halves = [torch.zeros(info.state_elems, device="cuda") for _ in range(2)]
    ws = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda")
    places = [[(0, 1), (511, (1 << 22) - 1), (512, 5), (1023, (1 << 22) - 2)], [(0, 0), (3, 9), (68, 63), (69, 62)]]
    for v, at in zip(g, places):
        for r, c in at:
            v[r, c] = 8.0
    Z.zero_muon_bind(h, None, None, [v.data_ptr() for v in x], [v.data_ptr() for v in g],
                     [v.data_ptr() for v in halves], ws.data_ptr(), 0, stream())
    Z.zero_muon_step(h, Z.muon_hyper(momentum=0.0, eps=1e-12, steps=1, coefficients=(1.5, -0.5, 0.0)), 1.0, stream())
    for v, at in zip(x, places):
        assert int(torch.count_nonzero(v)) == 4 and all(float(v[r, c]) == 0.5 * (1.5 - 0.125) for r, c in at)
    assert int(torch.count_nonzero(halves[1])) == 8
    torch.cuda.synchronize()
    Z.zero_muon_destroy(h)


# ------------------------------------------------------------------ with a sharded step

class Joined:
    def __init__(self, scaler=None):
        self.g = EmulatedGroup([4096, 300], 2, 2)
        for r in range(2):
            for _u, off, n, _b, _s in self.g.shard_slices(r):
                self.g.state[r]["master"][0][off:off + n] = 0.01
        n = int(self.g.info.max_contrib_elems)
        gen = torch.Generator().manual_seed(1)
        self.c = [(torch.randn(n, generator=gen) * 1e-2).to(torch.bfloat16).cuda() for _ in range(2)]
        self.mu = Muon([(64, 96), (130, 40)], 2, "bf16").fill(8)
        if scaler:
            Z.zero_set_scaler(self.g.plan, scaler, stream())

    def step(self, hyper, muon):
        plan, s = self.g.plan, stream()
        Z.zero_muon_check(self.mu.h, plan, muon, s)
        Z.zero_step(plan, [c.data_ptr() for c in self.c], -1, hyper, s)
        Z.zero_muon_step_with(self.mu.h, plan, muon, s)
        return Z.zero_step_finish(plan, s)

    def close(self):
        self.mu.close()
        self.g.close()


def test_joined_step():
    j, alone, muon = Joined(Z.scaler(scale=4.0)), Muon([(64, 96), (130, 40)], 2, "bf16").fill(8), Z.muon_hyper(lr=0.01)
    try:
        for k in range(2):
            assert j.step(Z.hyper(), muon).skipped == 0
            Z.zero_muon_step(alone.h, muon, 4.0, stream())
        assert all(torch.equal(a, b) for a, b in zip(alone.p + alone.halves, j.mu.p + j.mu.halves))
        # a matrix's gradient leaves out both
        kept = [v.clone() for v in j.mu.p + j.mu.x]
        good = j.mu.g[0][1][3, 3].clone()
        j.mu.g[0][1][3, 3] = float("inf")
        res = j.step(Z.hyper(), muon)
        assert res.skipped == 1 and res.scale == 2.0 and res.t == 2
        assert all(torch.equal(a, b) for a, b in zip(kept, j.mu.p + j.mu.x))
        assert Z.zero_muon_read(j.mu.h, stream()).skipped == 1
        # the plan's does so too
        j.mu.g[0][1][3, 3] = good
        good = j.c[1][7].clone()
        j.c[1][7] = float("nan")
        res = j.step(Z.hyper(), muon)
        assert res.skipped == 1 and res.scale == 1.0 and Z.zero_muon_read(j.mu.h, stream()).skipped_total == 2
        assert all(torch.equal(a, b) for a, b in zip(kept, j.mu.p + j.mu.x))
        j.c[1][7] = good
        Z.zero_muon_step(alone.h, muon, 1.0, stream())
        assert j.step(Z.hyper(), muon).t == 3
        assert all(torch.equal(a, b) for a, b in zip(alone.p, j.mu.p))
    finally:
        j.close()
        alone.close()


def test_joined_order():
    j, muon, s = Joined(), Z.muon_hyper(), stream()
    try:
        plan, h, ptrs = j.g.plan, j.mu.h, [c.data_ptr() for c in j.c]

        def refused(status, f, *args):
            with pytest.raises(Z.ZeroError) as e:
                f(*args)
            assert e.value.status == status

        refused(Z.ZERO_ESTATE, Z.zero_muon_step_with, h, plan, muon, s)
        Z.zero_muon_check(h, plan, muon, s)
        refused(Z.ZERO_ESTATE, Z.zero_muon_check, h, plan, muon, s)
        refused(Z.ZERO_ESTATE, Z.zero_muon_step_with, h, plan, muon, s)          # no bucket yet
        Z.zero_step(plan, ptrs, -1, Z.hyper(), s)
        refused(Z.ZERO_EINVAL, Z.zero_muon_step_with, h, plan, Z.muon_hyper(momentum=0.5), s)
        refused(Z.ZERO_EINVAL, Z.zero_muon_step_with, h, plan, Z.muon_hyper(nesterov=False), s)
        Z.zero_muon_step_with(h, plan, muon, s)
        refused(Z.ZERO_ESTATE, Z.zero_muon_step_with, h, plan, muon, s)
        assert Z.zero_step_finish(plan, s).t == 1
        # the matrices are no part of the plan's norm
        Z.zero_grad_norm(plan, ptrs, -1, s)
        Z.zero_muon_check(h, plan, muon, s)
        Z.zero_step(plan, ptrs, -1, Z.hyper(max_grad_norm=1e-3), s)
        Z.zero_muon_step_with(h, plan, muon, s)
        norm = Z.zero_step_finish(plan, s).grad_norm
        g = (j.c[0].double() + j.c[1].double())[:4396] / 2
        assert abs(norm - float(g.norm())) <= 1e-3 * norm
    finally:
        j.close()


def test_joined_order_after_a_step_or_a_bind():
    """What zero_muon_check formed is gone with a step of the handle's own or another bind."""
    j, muon, s = Joined(), Z.muon_hyper(), stream()
    try:
        plan, mu, ptrs = j.g.plan, j.mu, [c.data_ptr() for c in j.c]
        for spoil in (lambda: Z.zero_muon_step(mu.h, muon, 1.0, s), lambda: mu.bind(-1)):
            Z.zero_muon_check(mu.h, plan, muon, s)
            Z.zero_step(plan, ptrs, -1, Z.hyper(), s)
            spoil()
            with pytest.raises(Z.ZeroError) as e:
                Z.zero_muon_step_with(mu.h, plan, muon, s)
            assert e.value.status == Z.ZERO_ESTATE
            # it joins the step again
            Z.zero_muon_check(mu.h, plan, muon, s)
            Z.zero_muon_step_with(mu.h, plan, muon, s)
            Z.zero_step_finish(plan, s)
        assert Z.zero_muon_read(mu.h, s).t == 3
    finally:
        j.close()
