"""zero_muon where a few directions dominate, and the second of the two fp16 numbers that the first iterates are kept as.

Tolerances.  What carries the low part alone: with coefficients (a, 0, 0) and one or two steps X is a (or a a') times the
two numbers' sum.  Each time X is stored as two, their sum is within 2^-22 of it (2^-11 of what the first leaves, 2^-11 of
it); the norm behind X's scale has fp32 sums of at most 40 squares a thread and a few roundings more, 2^-19 in all.  The
first number alone is 2^-12 of X off and more at every second entry.

Accuracy: the float64 iteration is run with its operands rounded to fp16's 11 bits where the kernels round; the tolerance
is twice the norm by which that misses the unrounded iteration, and 2^-13 of the result for fp32 sums.  Of a rank-one
matrix with noise it is a third at most of what the iteration misses without the low part, which is checked too.
"""
import pytest
import torch
from test_gpu_muon import ABC, Muon, coefficients, expected, iterate, stream

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
# by the tiles that a handle of these matrices chooses, wide and tall; (two at once): where every side is at least 128
CUTS = {"128x64": [(96, 300), (300, 96)], "128x64, two at once": [(512, 512)],
        "128x128": [(2048, 1536), (60, 512)], "128x128, two at once": [(2048, 700)] * 2 + [(700, 2304)] * 3,
        "256x256": [(2304, 2100), (2100, 2304), (300, 90)], "256x256, two at once": [(2304, 2100)] + [(2100, 2304)] * 2}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def paired(shapes):
    return min(min(s) for s in shapes) >= 128


def rounded(v):
    """To 11 bits, ties to even."""
    m, e = torch.frexp(v)
    return torch.ldexp(torch.round(m * 2048) / 2048, e)


def fill(mu, make):
    """fp32 momentum of make(r, c), no gradients, no parameters."""
    for i, (r, c) in enumerate(mu.shapes):
        mu.m(0, i).copy_(make(r, c))
        mu.p[i].zero_()
        for g in mu.g:
            g[i].zero_()
    return mu


@pytest.mark.parametrize("a", [(1.0,), (1.5,), (1.0, 1.0), (1.25, 0.75)])
@pytest.mark.parametrize("name", sorted(CUTS))
def test_two_numbers_carry_x(name, a):
    gen = torch.Generator(device="cuda").manual_seed(1)
    mu = fill(Muon(CUTS[name], updates=False), lambda r, c: torch.randn(r, c, generator=gen, device="cuda"))
    try:
        hyper = Z.muon_hyper(lr=1.0, momentum=0.5, weight_decay=0.0, nesterov=False, scale=0, steps=len(a),
                             coefficients=[(v, 0.0, 0.0) for v in a])
        assert mu.step(hyper).t == 1
        for i in range(len(mu.shapes)):
            x = mu.m(0, i).double() / 2
            x = x / (x.norm() + hyper.eps)
            for v in a:
                x = x * v
            off = (mu.p[i].double() + x).abs()
            assert bool((off <= (len(a) * 2.0 ** -22 + 2.0 ** -19) * x.abs() + 2.0 ** -35).all()), float((off / x.abs()).max())
            alone = (rounded(x) - x).abs()
            assert float((alone > 2.0 ** -14 * x.abs()).double().mean()) > 0.5
    finally:
        mu.close()


def against_emulation(mu, hyper, pair, low_matters):
    want = [expected(mu, None, i, 0, hyper)[2] for i in range(len(mu.shapes))]
    assert mu.step(hyper).t == 1
    abc = coefficients(hyper)
    for i, u in enumerate(want):
        x = iterate(u, hyper.eps, abc)
        tol = 2 * float((iterate(u, hyper.eps, abc, rounded, pair) - x).norm()) + 2.0 ** -13 * float(x.norm())
        off = float((mu.p[i].double() + x).norm())
        assert off <= tol, (mu.shapes[i], off / float(x.norm()), tol / float(x.norm()))
        if low_matters:
            h = rounded(u / (u.norm() + hyper.eps))
            lost = float((iterate(h, 1.0 - float(h.norm()), abc, rounded, pair) - x).norm())
            assert lost > 3 * tol, (mu.shapes[i], lost / float(x.norm()), tol / float(x.norm()))


USUAL = dict(lr=1.0, weight_decay=0.0, scale=0, coefficients=ABC)


@pytest.mark.parametrize("name", sorted(CUTS))
def test_rank_one_and_noise(name):
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda r, c: torch.randn(r, c, generator=gen, device="cuda")  # noqa: E731
    mu = fill(Muon(CUTS[name], updates=False), lambda r, c: new(r, 1) @ new(1, c) + 0.01 * new(r, c))
    try:
        against_emulation(mu, Z.muon_hyper(**USUAL), paired(CUTS[name]), True)
    finally:
        mu.close()


@pytest.mark.parametrize("name", sorted(CUTS))
def test_dense(name):
    """Tall and wide ones on each of the tiles, to twice the roundings' own error."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    mu = fill(Muon(CUTS[name], updates=False), lambda r, c: torch.randn(r, c, generator=gen, device="cuda"))
    try:
        against_emulation(mu, Z.muon_hyper(**USUAL), paired(CUTS[name]), False)
    finally:
        mu.close()


@pytest.mark.parametrize("shape,rows", [((3, 512), 3), ((4, 512), 4), ((32, 512), 32), ((256, 512), 1), ((256, 512), 4),
                                        ((256, 512), 8), ((512, 256), 4)])
def test_few_rows(shape, rows):
    """Few singular values, which the rows that are not zero have all of: the roundings' error is largest here, about 1 % of
    the result."""
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def make(r, c):
        v = torch.zeros(r, c, device="cuda")
        if r >= rows and r <= c:
            v[:rows] = torch.randn(rows, c, generator=gen, device="cuda")
        else:
            v[:, :rows] = torch.randn(r, rows, generator=gen, device="cuda")
        return v

    mu = fill(Muon([shape], updates=False), make)
    try:
        want = expected(mu, None, 0, 0, Z.muon_hyper(**USUAL))[2]
        x = iterate(want, 1e-7, [ABC] * 5)
        against_emulation(mu, Z.muon_hyper(**USUAL), paired([shape]), False)
        off = torch.linalg.matrix_norm(mu.p[0].double() + x, 2) / torch.linalg.matrix_norm(x, 2)
        assert float(off) < 0.015, float(off)
    finally:
        mu.close()


def test_streams_share_nothing():
    """The same matrices twice at once: the low parts lie in a workspace of each handle."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    made = torch.randn(96, 1, generator=gen, device="cuda") @ torch.randn(1, 300, generator=gen, device="cuda")
    made = made + 0.01 * torch.randn(96, 300, generator=gen, device="cuda")
    ref, *both = (fill(Muon([(96, 300)], updates=False), lambda r, c: made) for _ in range(3))
    hyper = Z.muon_hyper(**USUAL)
    try:
        ref.step(hyper)
        streams = [torch.cuda.Stream() for _ in both]
        for mu, s in zip(both, streams):
            Z.zero_muon_step(mu.h, hyper, 1.0, s.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(ref.p[0], mu.p[0]) and Z.zero_muon_read(mu.h, stream()).t == 1 for mu in both)
    finally:
        for mu in (ref, *both):
            mu.close()
