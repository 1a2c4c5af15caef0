"""zero_gated and its gradients against float64.

Tolerances.  u16 = 2^-8 (bf16) or 2^-11 (fp16) is one rounding of a 16-bit output, and of dg and du before the
products of the gradient; below 2^-14 an fp16 rounding is 2^-25 instead.  A product's sum has one rounded (at worst
truncated, 2^-23) addition for every 16 inner elements, one more for a bias or an old gradient: at most
(K / 16 + 80) 2^-23 of the sum of magnitudes.  The activations' fp32 values are within 2^-19 of |z| + 1 and their
slopes, at most 1.2, within 2^-17.  A bias's sum has at most one rounding for each row.  Whole numbers whose sums
stay below 2^24 are exact.
"""
import pytest
import torch
from test_gpu_linear import ACTS, DTYPES, act64, matrix, storage, untouched

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -25


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def call(args, back, stream=None):
    n = Z.zero_gated_workspace(args, back)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    stream = stream or torch.cuda.current_stream()
    (Z.zero_gated_backward if back else Z.zero_gated)(args, ws.data_ptr(), n, stream.cuda_stream)
    return ws


def product_error(inner, mag):
    return (inner / 16 + 80) * 2.0 ** -23 * mag


class Block:
    def __init__(self, m, k, n, dtype="bf16", layout="out_in", act="silu", bias=True, keep=True, whole=False, pad=0,
                 shift=0, seed=0):
        t, kind, self.u16 = DTYPES[dtype]
        gen = torch.Generator().manual_seed(seed)
        self.m, self.k, self.n, self.act, self.t, self.layout = m, k, n, act, t, layout
        new = lambda r, c, std=1.0: matrix(r, c, t, gen, c + pad, shift, whole, std)  # noqa: E731
        weight = lambda: new(n, k, max(k, 1) ** -0.5) if layout == "out_in" else new(k, n, max(k, 1) ** -0.5)  # noqa: E731
        self.x, self.w_gate, self.w_up = new(m, k), weight(), weight()
        self.b_gate, self.b_up = (new(1, n), new(1, n)) if bias else (None, None)
        self.h, self.gate, self.up, self.dh = new(m, n), new(m, n), new(m, n), new(m, n)
        self.dx, self.dw_gate, self.dw_up, self.db_gate, self.db_up = new(m, k), weight(), weight(), new(1, n), new(1, n)
        cols = self.w_gate.shape[1] + pad
        self.args = Z.zero_gated_t(
            rows=m, in_features=k, out_features=n, dtype16=kind, activation=ACTS[act],
            layout=Z.ZERO_WEIGHT_OUT_IN if layout == "out_in" else Z.ZERO_WEIGHT_IN_OUT, ld_x=k + pad, ld_w_gate=cols,
            ld_w_up=cols, ld_h=n + pad, ld_gate=n + pad, ld_up=n + pad, ld_dh=n + pad, ld_dx=k + pad, ld_dw_gate=cols,
            ld_dw_up=cols)
        for name in ("x", "w_gate", "w_up", "b_gate", "b_up", "h", "gate", "up", "dh", "dx", "dw_gate", "dw_up",
                     "db_gate", "db_up"):
            v = getattr(self, name)
            if v is not None and (keep or name not in ("gate", "up")):
                setattr(self.args, name, v.data_ptr())

    def weights64(self):
        return [(w.t() if self.layout == "out_in" else w).double() for w in (self.w_gate, self.w_up)]   # (in, out)

    def check_forward(self, exact=False):
        names = [k for k in ("h", "gate", "up") if getattr(self.args, k)]
        before = {k: storage(getattr(self, k)) for k in ("h", "gate", "up")}
        call(self.args, False)
        for name in before:
            if name in names:
                untouched(getattr(self, name), before[name])
            else:
                assert torch.equal(storage(getattr(self, name)), before[name])
        x, z, e = self.x.double(), [], []
        for w, b in zip(self.weights64(), (self.b_gate, self.b_up)):
            b = b.double() if b is not None else torch.zeros((), dtype=torch.float64, device="cuda")
            z.append(x @ w + b)
            e.append(product_error(self.k, x.abs() @ w.abs() + b.abs()))
        a = act64(z[0], self.act)
        h = a * z[1]
        for name, want, err in (("gate", z[0], e[0]), ("up", z[1], e[1]),
                                ("h", h, z[1].abs() * (1.2 * e[0] + 2.0 ** -19 * (z[0].abs() + 1) * (self.act != "none"))
                                 + a.abs() * e[1] + 2 * e[0] * e[1] + 2.0 ** -23 * h.abs())):
            if name not in names:
                continue
            got = getattr(self, name)
            if exact:
                assert torch.equal(got, want.to(self.t)), name
                continue
            bound = err + self.u16 * want.abs() + TINY
            off = (got.double() - want).abs()
            assert bool((off <= bound).all()), (name, float((off / bound).max()))

    def gradients64(self):
        """dg, du and the bounds of their errors, rounded to 16 bits and before that."""
        g = self.gate.double().requires_grad_(True)
        u, d = self.up.double(), self.dh.double()
        a = act64(g, self.act)
        slope = torch.autograd.grad(a.sum(), g)[0] if self.act != "none" else torch.ones_like(u)
        a, g = a.detach(), g.detach()
        dg, du = d * u * slope, d * a
        fine = (0.0, 0.0) if self.act in ("none", "relu") else (2.0 ** -17, 2.0 ** -19)
        eg = (d * u).abs() * fine[0] + 2.0 ** -22 * dg.abs()
        eu = d.abs() * (g.abs() + 1) * fine[1] + 2.0 ** -23 * du.abs()
        return (dg, du), (eg, eu), [e + self.u16 * v.abs() + TINY for e, v in ((eg, dg), (eu, du))]

    def check_backward(self, exact=False, accumulate=False):
        names = [k for k in ("dx", "dw_gate", "dw_up", "db_gate", "db_up") if getattr(self.args, k)]
        before = {k: storage(getattr(self, k)) for k in names}
        old = {k: getattr(self, k).double().clone() for k in names}
        self.args.flags = Z.ZERO_GATED_ACCUMULATE if accumulate else 0
        call(self.args, True)
        x, w = self.x.double(), self.weights64()
        dz, fine, rough = self.gradients64()
        for name in names:
            if name == "dx":
                want = sum(d @ v.t() for d, v in zip(dz, w))
                err = sum(r @ v.abs().t() for r, v in zip(rough, w))
                err = err + product_error(2 * self.n, sum(d.abs() @ v.abs().t() for d, v in zip(dz, w)))
            else:
                i = name.endswith("up")
                if name.startswith("dw"):
                    pair = (lambda d: d.t() @ x) if self.layout == "out_in" else (lambda d: x.t() @ d)
                    big = (lambda d: d.t() @ x.abs()) if self.layout == "out_in" else (lambda d: x.abs().t() @ d)
                    want, err = pair(dz[i]), big(rough[i]) + product_error(self.m, big(dz[i].abs()))
                else:
                    want = dz[i].sum(0, keepdim=True)
                    err = fine[i].sum(0) + (self.m + 8) * 2.0 ** -24 * dz[i].abs().sum(0)
                if accumulate:
                    want = want + old[name]
                    err = err + 2.0 ** -23 * (want.abs() + old[name].abs())
            got = getattr(self, name)
            untouched(got, before[name])
            if exact:
                assert torch.equal(got, want.to(self.t)), name
                continue
            bound = err + self.u16 * want.abs() + TINY
            off = (got.double() - want).abs()
            assert bool((off <= bound).all()), (name, float((off / bound).max()))


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", [(1, 64, 64), (1, 520, 72), (2, 2048, 1000), (1, 8, 8), (2, 264, 4096), (1, 1001, 77),
                                   (3, 64, 128), (24, 200, 136), (129, 72, 65), (300, 1001, 130), (640, 256, 1280),
                                   (257, 65, 1603)])
def test_forward(m, k, n, layout):
    for i, act in enumerate(("silu", "gelu_tanh")):
        Block(m, k, n, ("bf16", "fp16")[i], layout, act, bias=i == 0, keep=i == 0, seed=m + n).check_forward()


@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("dtype", sorted(DTYPES))
def test_activations(act, dtype):
    for m in (1, 2, 40):
        Block(m, 96, 136, dtype, "in_out", act, seed=m).check_forward()
    Block(40, 96, 136, dtype, "out_in", act, seed=3).check_backward()


@pytest.mark.parametrize("pad,shift", [(8, 8), (8, 0), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_strides(pad, shift, layout):
    for m in (1, 2, 70, 300):
        b = Block(m, 128, 200, "bf16", layout, pad=pad, shift=shift, seed=m)
        b.check_forward()
        b.check_backward()
        b.check_backward(accumulate=True)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", [(1, 64, 64), (3, 1, 1), (24, 200, 136), (129, 72, 65), (300, 1001, 130),
                                   (640, 256, 1280), (1000, 640, 257), (2, 8, 1603)])
def test_backward(m, k, n, layout):
    for i, act in enumerate(("silu", "gelu")):
        Block(m, k, n, ("bf16", "fp16")[i], layout, act, seed=m + n).check_backward(accumulate=i == 1)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", [(40, 4096, 72), (130, 5000, 130), (300, 96, 5000), (129, 70, 6400), (4000, 72, 136),
                                   (2500, 130, 64), (6000, 64, 2000)])
def test_few_tiles_and_a_long_sum(m, k, n, layout):
    """Parts of the inner dimension as tiles of their own, of one product or of two; narrow and wide columns' sums."""
    for pad in (0, 8, 3):
        b = Block(m, k, n, "bf16", layout, pad=pad, seed=k)
        b.check_forward()
        b.check_backward()
    b.check_backward(accumulate=True)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", [(16, 4096, 9856), (140, 4096, 4900), (500, 8192, 4992), (1000, 4160, 2500)])
def test_tiles_past_a_full_round(m, k, n, layout):
    """Whole tiles, and the few that would not fill a round of the SMs in parts."""
    for pad, keep in ((0, True), (3, False)):
        Block(m, k, n, "bf16", layout, pad=pad, keep=keep, seed=k).check_forward()


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_whole_numbers_are_exact(layout):
    for act in ("none", "relu"):
        for m, k, n in ((1, 64, 72), (2, 512, 64), (200, 96, 300), (513, 64, 520), (130, 64, 4000)):
            b = Block(m, k, n, "bf16", layout, act, whole=True, seed=k)
            b.check_forward(exact=k <= 64)
            b = Block(m, k, n, "bf16", layout, act, whole=True, seed=k)      # dg, du: whole numbers of at most 4
            b.check_backward(exact=True)
            b.check_backward(exact=False, accumulate=True)


def test_some_gradients_only():
    for wanted in (("dx",), ("dw_up",), ("dw_gate",), ("db_up",), ("db_gate", "dx"), ("dw_gate", "dw_up")):
        b = Block(70, 72, 136, seed=1)
        for name in ("dx", "dw_gate", "dw_up", "db_gate", "db_up"):
            if name not in wanted:
                setattr(b.args, name, None)
        left = {k: storage(getattr(b, k)) for k in ("dx", "dw_gate", "dw_up", "db_gate", "db_up") if k not in wanted}
        b.check_backward()
        for k, v in left.items():
            assert torch.equal(storage(getattr(b, k)), v)


def test_empty_sizes():
    b = Block(0, 64, 72)
    call(b.args, False)
    b.check_backward()
    b = Block(0, 64, 72)
    old = b.dw_gate.clone()
    b.args.flags = Z.ZERO_GATED_ACCUMULATE
    call(b.args, True)
    assert torch.equal(old, b.dw_gate)
    b = Block(5, 0, 72)
    b.check_forward()
    b.args.dx = b.args.dw_gate = b.args.dw_up = None
    b.check_backward()
    b = Block(5, 64, 0)
    call(b.args, False)
    b.check_backward()


@pytest.mark.parametrize("m", [1, 2, 5, 140])
def test_a_row_that_is_not_finite_stays_alone(m):
    for bad in (float("inf"), float("nan")):
        b = Block(m, 136, 200, seed=m)
        call(b.args, False)
        kept = b.h.clone()
        b.x[m - 1, 3] = bad
        call(b.args, False)
        assert torch.equal(kept[:m - 1], b.h[:m - 1]) and not bool(torch.isfinite(b.h[m - 1]).any())


def test_gradient_against_differences():
    b = Block(60, 72, 136, "fp16", "in_out", "gelu", seed=4)
    call(b.args, False)
    call(b.args, True)
    names = ("x", "w_gate", "w_up", "b_gate", "b_up")
    at = {k: getattr(b, k).double() for k in names}
    dh, wg, wu, x = b.dh.double(), *b.weights64(), at["x"].abs()
    # roundings of g and u as kept (each moves dg and du by at most that share of these), of dg and du, and of the
    # result: three of 2^-11 and the fp32 sums' few 2^-20
    g, u = b.gate.double().abs(), b.up.double().abs()
    big_g, big_u = dh.abs() * u * (1.2 + g), dh.abs() * (1.2 + g)
    big = {"x": big_g @ wg.abs().t() + big_u @ wu.abs().t(), "w_gate": x.t() @ big_g, "w_up": x.t() @ big_u,
           "b_gate": big_g.sum(0, keepdim=True), "b_up": big_u.sum(0, keepdim=True)}
    for name in names:
        v = getattr(b, "d" + name).double()              # along the gradient itself, where the difference is largest
        v = v / v.norm()

        def loss(step):
            p = dict(at)
            p[name] = at[name] + step * v
            g, u = p["x"] @ p["w_gate"] + p["b_gate"], p["x"] @ p["w_up"] + p["b_up"]
            return float((dh * act64(g, "gelu") * u).sum())

        want, got = (loss(1e-4) - loss(-1e-4)) / 2e-4, float((getattr(b, "d" + name).double() * v).sum())
        assert abs(got - want) <= 3.1 * 2.0 ** -11 * float((big[name] * v.abs()).sum()) + 1e-6, name


@pytest.mark.parametrize("m,k,n", [(90, 136, 200), (40, 4096, 72), (130, 70, 6400)])
def test_streams_and_graphs(m, k, n):
    b = Block(m, k, n, "bf16", "in_out", pad=1, seed=5)            # rows off the 16-byte grid: copies as well
    call(b.args, False)
    call(b.args, True)
    torch.cuda.synchronize()
    names = ("h", "gate", "up", "dx", "dw_gate", "dw_up", "db_gate", "db_up")
    want = {k: getattr(b, k).clone() for k in names}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ws = [call(b.args, False, side), call(b.args, True, side)]
    side.synchronize()
    assert all(torch.equal(want[k], getattr(b, k)) for k in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stream = torch.cuda.current_stream().cuda_stream
        Z.zero_gated(b.args, ws[0].data_ptr(), ws[0].numel(), stream)
        Z.zero_gated_backward(b.args, ws[1].data_ptr(), ws[1].numel(), stream)
    for _ in range(3):
        for k in names:
            getattr(b, k).zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], getattr(b, k)) for k in names)


@pytest.mark.parametrize("m,k,n", [(500, 1024, 1100), (40, 4096, 72), (3000, 70, 6400)])
def test_repeats_are_the_same_bits(m, k, n):
    b = Block(m, k, n, seed=6)
    out = []
    for _ in range(3):
        call(b.args, False)
        call(b.args, True)
        out.append([getattr(b, k).clone() for k in ("h", "dx", "dw_gate", "dw_up", "db_gate")])
    assert all(torch.equal(p, q) for o in out[1:] for p, q in zip(out[0], o))
