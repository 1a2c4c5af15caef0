"""zero_linear and its gradients against float64.

Tolerances.  u16 = 2^-8 (bf16) or 2^-11 (fp16) is one rounding of a 16-bit output, and of dz before
the two products of the gradient; below 2^-14 an fp16 rounding is 2^-25 instead.  A product's sum has one rounded (at worst truncated, 2^-23)
addition for every 16 inner elements, one more for every split, bias and residual: at most
(K / 16 + 80) 2^-23 of the sum of magnitudes.  The activations' slopes are at most 1.2 and their
fp32 values within 2^-19 of |z| + 1.  Whole numbers whose sums stay below 2^24 are exact.
"""
import math

import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
ACTS = {"none": Z.ZERO_ACT_NONE, "relu": Z.ZERO_ACT_RELU, "gelu_tanh": Z.ZERO_ACT_GELU_TANH,
        "gelu": Z.ZERO_ACT_GELU, "silu": Z.ZERO_ACT_SILU}
DTYPES = {"bf16": (torch.bfloat16, Z.ZERO_BF16, 2.0 ** -8), "fp16": (torch.float16, Z.ZERO_FP16, 2.0 ** -11)}
GUARD = 5.0


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def matrix(rows, cols, dtype, gen, ld=0, shift=0, whole=False, std=1.0):
    """A rows x cols view with row stride ld, `shift` elements into its storage."""
    ld = max(ld, cols)
    buf = torch.full((rows * ld + shift + 16,), GUARD, dtype=dtype, device="cuda")
    v = torch.as_strided(buf, (rows, cols), (ld, 1), shift)
    if whole:
        v.copy_(torch.randint(-2, 3, (rows, cols), generator=gen).to(dtype))
    else:
        v.copy_((torch.randn(rows, cols, generator=gen) * std).to(dtype))
    return v


def untouched(v, before):
    """Storage outside a view is as it was."""
    buf = torch.as_strided(v, (v.untyped_storage().nbytes() // v.element_size(),), (1,), 0)
    mask = torch.ones_like(buf, dtype=torch.bool)
    torch.as_strided(mask, v.shape, v.stride(), v.storage_offset()).fill_(False)
    assert torch.equal(buf[mask].view(torch.int16), before[mask].view(torch.int16))


def storage(v):
    return torch.as_strided(v, (v.untyped_storage().nbytes() // v.element_size(),), (1,), 0).clone()


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)          # its slope at 0 is 0
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2))
    return z * torch.sigmoid(z) if act == "silu" else z


def workspace(args, back):
    n = Z.zero_linear_workspace(args, back)
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda"), n


def call(args, back):
    ws, n = workspace(args, back)
    (Z.zero_linear_backward if back else Z.zero_linear)(args, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    return ws


class Layer:
    def __init__(self, m, k, n, dtype="bf16", layout="out_in", act="none", bias=True, residual=True, whole=False,
                 pad=0, shift=0, seed=0):
        t, self.kind, self.u16 = DTYPES[dtype]
        gen = torch.Generator().manual_seed(seed)
        self.m, self.k, self.n, self.act, self.t, self.layout = m, k, n, act, t, layout
        new = lambda r, c, std=1.0: matrix(r, c, t, gen, c + pad, shift, whole, std)  # noqa: E731
        self.x = new(m, k)
        self.w = new(n, k, max(k, 1) ** -0.5) if layout == "out_in" else new(k, n, max(k, 1) ** -0.5)
        self.bias = new(1, n) if bias else None
        self.residual = new(m, n) if residual else None
        self.y, self.pre, self.dy = new(m, n), new(m, n), new(m, n)
        self.dx, self.dw, self.dbias = new(m, k), new(*self.w.shape), new(1, n)
        self.args = Z.zero_linear_t(
            rows=m, in_features=k, out_features=n, dtype16=self.kind,
            layout=Z.ZERO_WEIGHT_OUT_IN if layout == "out_in" else Z.ZERO_WEIGHT_IN_OUT, activation=ACTS[act],
            ld_x=k + pad, ld_w=self.w.shape[1] + pad, ld_y=n + pad, ld_pre=n + pad, ld_residual=n + pad,
            ld_dy=n + pad, ld_dx=k + pad, ld_dw=self.w.shape[1] + pad)
        for name in ("x", "w", "bias", "residual", "y", "pre", "dy", "dx", "dw", "dbias"):
            v = getattr(self, name)
            setattr(self.args, name, v.data_ptr() if v is not None else None)

    def matrix_w(self):
        return (self.w.t() if self.layout == "out_in" else self.w).double()     # (in, out)

    def forward64(self):
        """z, y and a bound of z's fp32 error."""
        x, w = self.x.double(), self.matrix_w()
        z, mag = x @ w, x.abs() @ w.abs()
        if self.bias is not None:
            z, mag = z + self.bias.double(), mag + self.bias.double().abs()
        y = act64(z, self.act)
        if self.residual is not None:
            y, mag = y + self.residual.double(), mag + self.residual.double().abs()
        return z, y, (self.k / 16 + 80) * 2.0 ** -23 * mag + 2.0 ** -149

    def slope64(self):
        z = self.pre.double().requires_grad_(True)
        return torch.autograd.grad(act64(z, self.act).sum(), z)[0] if self.act != "none" else torch.ones_like(z)

    def check_forward(self, exact=False):
        before = {k: storage(getattr(self, k)) for k in ("y", "pre")}
        residual = self.residual.clone() if self.residual is not None else None
        call(self.args, False)
        z, y, dz = self.forward64()
        assert residual is None or torch.equal(residual, self.residual)
        for name in before:
            untouched(getattr(self, name), before[name])
        if exact:
            assert torch.equal(self.pre, z.to(self.t)) and torch.equal(self.y, y.to(self.t))
            return
        assert bool(((self.pre.double() - z).abs() <= dz + self.u16 * z.abs() + 2.0 ** -25).all())
        bound = 1.2 * dz + 2.0 ** -19 * (z.abs() + 1) * (self.act != "none") + self.u16 * y.abs() + 2.0 ** -25
        err = (self.y.double() - y).abs()
        assert bool((err <= bound).all()), float((err / bound).max())

    def check_backward(self, exact=False, accumulate=False):
        names = [k for k in ("dx", "dw", "dbias") if getattr(self.args, k)]
        before = {k: storage(getattr(self, k)) for k in names}
        old = {k: getattr(self, k).double().clone() for k in names}
        self.args.flags = Z.ZERO_LINEAR_ACCUMULATE if accumulate else 0
        call(self.args, True)
        x, w, dz = self.x.double(), self.matrix_w(), self.dy.double() * self.slope64()
        rounded = 0.0 if exact else self.u16 + 2.0 ** -18 * (self.act != "none")      # dz's own rounding
        for name in names:
            if name == "dx":
                want, mag, inner = dz @ w.t(), dz.abs() @ w.abs().t(), self.n
                low = 2.0 ** -25 * w.abs().sum(1)
            elif name == "dw":
                a, b = (dz, x) if self.layout == "out_in" else (x, dz)
                want, mag, inner = a.t() @ b, a.abs().t() @ b.abs(), self.m
                low = 2.0 ** -25 * x.abs().sum(0)
                low = low[None, :] if self.layout == "out_in" else low[:, None]
            else:
                want, mag, inner = dz.sum(0, keepdim=True), dz.abs().sum(0, keepdim=True), 16 * self.m
                low = 0.0
            if accumulate and name != "dx":
                want, mag = want + old[name], mag + old[name].abs()
            got = getattr(self, name).double()
            untouched(getattr(self, name), before[name])
            if exact:
                assert torch.equal(getattr(self, name), want.to(self.t)), name
            else:
                bound = ((inner / 16 + 80) * 2.0 ** -23 + rounded) * mag + low + self.u16 * want.abs() + 2.0 ** -25
                assert bool(((got - want).abs() <= bound).all()), (name, float(((got - want).abs() / bound).max()))


SHAPES = [(1, 64, 128), (1, 1, 1), (3, 5, 7), (1, 1000, 513), (2, 256, 2048), (16, 512, 96), (17, 130, 300), (129, 65, 257),
          (128, 64, 128), (256, 256, 256), (300, 1024, 520), (513, 192, 1000), (1000, 72, 40), (64, 4096, 64)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_whole_numbers_are_exact(shape, layout, dtype):
    """Every element of every product in its place: whole numbers have one answer."""
    layer = Layer(*shape, dtype=dtype, layout=layout, act="relu", whole=True, seed=sum(shape))
    layer.check_forward(exact=True)
    layer.check_backward(exact=True)
    layer.check_backward(exact=True, accumulate=True)


@pytest.mark.parametrize("pad,shift", [(0, 1), (8, 0), (8, 8), (3, 0), (1, 5)])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
def test_strides_and_starts(pad, shift, layout):
    for shape in ((70, 136, 264), (5, 129, 33)):
        layer = Layer(*shape, layout=layout, act="relu", whole=True, pad=pad, shift=shift, seed=pad + shift)
        layer.check_forward(exact=True)
        layer.check_backward(exact=True)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bias,residual", [(True, True), (False, False)])
def test_activations(act, dtype, bias, residual):
    for shape, layout in (((1, 640, 384), "in_out"), ((200, 320, 448), "out_in"), ((77, 101, 163), "in_out"),
                          ((1, 77, 131), "out_in")):
        layer = Layer(*shape, dtype=dtype, layout=layout, act=act, bias=bias, residual=residual, seed=3)
        layer.check_forward()
        if not bias:
            layer.args.dbias = None
        layer.check_backward()
        layer.check_backward(accumulate=True)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("rows", [1, 2, 4, 7, 8, 9, 16, 31, 64, 100, 128])
def test_few_rows(rows, layout):
    layer = Layer(rows, 2048, 1024, layout=layout, act="gelu_tanh", seed=rows)
    layer.check_forward()
    layer.check_backward()


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("inner,outer", [(8, 8), (8, 1000), (248, 72), (256, 1), (264, 24), (520, 3000), (1032, 6), (2056, 19464),
                                         (2040, 8), (4104, 136), (8184, 2056), (30000, 64)])
def test_one_and_two_rows(rows, layout, inner, outer):
    """Parts of the inner dimension that end anywhere, columns and rows of the weight that do not fill a block."""
    for dtype, pad in (("bf16", 0), ("fp16", 8)):
        layer = Layer(rows, inner, outer, dtype=dtype, layout=layout, act="relu", whole=True, pad=pad, seed=inner + outer)
        layer.check_forward(exact=True)
        layer.x[-1, inner // 2] = float("inf")        # the last row's own, and no other's
        first = layer.y[: rows - 1].clone()
        call(layer.args, False)
        assert torch.equal(layer.y[: rows - 1], first)
        want = layer.matrix_w()[inner // 2] * float("inf")
        assert torch.equal(layer.pre[-1].double().nan_to_num(0.0, 1.0, -1.0)[want != 0], want[want != 0].clamp(-1, 1).nan_to_num(0.0))


def test_split_inner_dimension():
    """Few tiles over a long inner dimension, in each of the three products."""
    for shape in ((64, 16384, 128), (64, 128, 16384), (16384, 64, 128)):
        layer = Layer(*shape, act="silu", seed=9)
        layer.check_forward()
        layer.check_backward(accumulate=True)


def test_many_tiles():
    layer = Layer(2500, 1088, 5000, layout="in_out", act="gelu", seed=2)
    layer.check_forward()
    layer.check_backward()


@pytest.mark.parametrize("act", list(ACTS))
def test_gradients_are_the_differences(act):
    """<gradient, direction> against central differences of the float64 forward."""
    layer = Layer(60, 48, 72, dtype="fp16", act=act, seed=4)
    x, w = layer.x.double(), layer.matrix_w()
    z = x @ w + layer.bias.double()
    layer.pre.copy_(z.to(layer.t))
    layer.dy.copy_(layer.dy.abs().to(layer.t) * 0.5 + 0.1)      # no cancellation over the outputs
    call(layer.args, True)
    dy, gen = layer.dy.double(), torch.Generator().manual_seed(1)
    grads = {"x": layer.dx.double(), "w": (layer.dw.t() if layer.layout == "out_in" else layer.dw).double(),
             "b": layer.dbias.double()}
    at = {"x": x, "w": w, "b": layer.bias.double()}
    for name in at:
        d = grads[name].sign()                                  # the direction with the largest change
        step = 1e-5 if act != "relu" else 1e-7
        value = []
        for s in (step, -step):
            v = {k: a + s * d if k == name else a for k, a in at.items()}
            value.append(float((act64(v["x"] @ v["w"] + v["b"], act) * dy).sum()))
        want, got = (value[0] - value[1]) / (2 * step), float((grads[name] * d).sum())
        # the gradient's own roundings (its 16 bits, dz's, and pre's through a slope that changes
        # by at most 1.1 a unit), all of one sign at worst; a relu's kink may be crossed
        assert abs(got - want) <= 2.0 ** -8 * abs(want), (name, got, want)


def test_y_over_residual_and_missing_outputs():
    layer = Layer(150, 96, 136, act="relu", whole=True)
    _, want, _ = layer.forward64()
    layer.args.y, layer.args.pre = layer.args.residual, None
    call(layer.args, False)
    assert torch.equal(layer.residual, want.to(layer.t))
    for only in ("dx", "dw", "dbias"):
        layer = Layer(150, 96, 136, act="relu", whole=True)
        for name in ("dx", "dw", "dbias"):
            if name != only:
                setattr(layer.args, name, None)
        layer.check_backward(exact=True)


@pytest.mark.parametrize("m,k,n", [(0, 8, 8), (8, 0, 24), (8, 8, 0), (1, 0, 1)])
def test_empty_sizes(m, k, n):
    layer = Layer(m, k, n, act="relu", whole=True)
    layer.check_forward(exact=True)
    layer.check_backward(exact=True)
    layer.check_backward(exact=True, accumulate=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(dtype):
    layer = Layer(200, 72, 136, dtype=dtype, act="none", residual=False, bias=False)
    layer.x[3, 5], layer.x[190, 71] = math.inf, math.nan
    call(layer.args, False)
    bad = ~torch.isfinite(layer.y)
    assert bool(bad[3].all()) and bool(bad[190].all()) and int(bad.sum()) == 2 * 136
    # a sum beyond the largest fp16 rounds to infinity
    if dtype == "fp16":
        layer = Layer(20, 72, 136, dtype=dtype, bias=False, residual=False)
        layer.x.fill_(200.0)
        layer.w.fill_(200.0)
        call(layer.args, False)
        assert bool(torch.isinf(layer.y).all())


def test_another_stream_and_a_graph():
    layer = Layer(300, 128, 264, layout="in_out", act="gelu")
    side = torch.cuda.Stream()
    ws, n = workspace(layer.args, False)
    wb, nb = workspace(layer.args, True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        Z.zero_linear(layer.args, ws.data_ptr(), n, side.cuda_stream)
        Z.zero_linear_backward(layer.args, wb.data_ptr(), nb, side.cuda_stream)
    torch.cuda.synchronize()
    want = [t.clone() for t in (layer.y, layer.pre, layer.dx, layer.dw, layer.dbias)]
    for t in (layer.y, layer.dx, layer.dw, layer.dbias):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream().cuda_stream
        Z.zero_linear(layer.args, ws.data_ptr(), n, s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(layer.y, want[0])
    Z.zero_linear_backward(layer.args, wb.data_ptr(), nb, torch.cuda.current_stream().cuda_stream)
    # pre has been written anew with the same values
    for got, w in zip((layer.y, layer.pre, layer.dx, layer.dw, layer.dbias), want):
        assert torch.equal(got, w)


def test_a_short_workspace_is_refused_before_anything_runs():
    layer = Layer(16, 4099, 33)
    n = Z.zero_linear_workspace(layer.args, True)
    assert n > 0
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    before = layer.dx.clone()
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_linear_backward(layer.args, ws.data_ptr(), n - 1)
    assert e.value.status == Z.ZERO_ERANGE
    assert torch.equal(before, layer.dx)
