"""zero_block_norm and its gradients against float64.

Tolerances.  u16 = 2^-8 (bf16) or 2^-11 (fp16, 2^-25 below 2^-14) is one rounding of an output, u = 2^-24 one of fp32.  A sum over a row is
a tree of at most 8 + 10 additions of terms with a few roundings each; centring loses (|a| + |mean|)
r in front of the normalised a, r = 1 / std.  64 u of those magnitudes covers a normalised row, 256 u
a gradient that goes through one (two such rows, their products and sums).  Sums over n rows add
n + 64 roundings of the terms' magnitudes.
"""
import math

import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": (torch.bfloat16, Z.ZERO_BF16, 2.0 ** -8), "fp16": (torch.float16, Z.ZERO_FP16, 2.0 ** -11)}
U = 2.0 ** -24
GUARD = 5.0
VECTORS = ("post_w", "post_b", "pre_w", "pre_b")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


def storage(v):
    return torch.as_strided(v, (v.untyped_storage().nbytes() // v.element_size(),), (1,), 0)


class Norm:
    def __init__(self, rows, dim, dtype="bf16", layer=False, post=True, pre=True, gate_rows=1, pad=0, shift=0, bias=None,
                 x=True, scale=0.7, eps=1e-5, mean=0.0, seed=0):
        self.t, self.kind, self.u16 = DTYPES[dtype]
        gen = torch.Generator().manual_seed(seed)
        self.rows, self.dim, self.layer, self.post, self.pre = rows, dim, layer, post, pre
        self.gate_rows, self.scale, self.eps = gate_rows, scale, eps
        groups = -(-rows // gate_rows) if gate_rows else 0
        bias = layer if bias is None else bias
        self.v = {}

        def new(name, r, c, there=True, std=1.0, mean=0.0):
            if not there:
                return
            buf = torch.full((r * (c + pad) + shift + 16,), GUARD, dtype=self.t, device="cuda")
            v = torch.as_strided(buf, (r, c), (c + pad, 1), shift)
            v.copy_((torch.randn(r, c, generator=gen) * std + mean).to(self.t))
            self.v[name] = v

        new("h", rows, dim, mean=mean)
        new("x", rows, dim, x, 2.0)
        new("gate", groups, dim, gate_rows > 0, 0.5, 0.5)
        new("post_w", 1, dim, post, 0.1, 1.0)
        new("post_b", 1, dim, post and bias, 0.1)
        new("pre_w", 1, dim, pre, 0.1, 1.0)
        new("pre_b", 1, dim, pre and bias, 0.1)
        for name in ("y", "z", "dy", "dz", "dx", "dh"):
            new(name, rows, dim, name not in ("z", "dz") or pre, mean=mean if name == "y" else 0.0)
        new("dgate", groups, dim, gate_rows > 0)
        for name in VECTORS:
            new("d" + name, 1, dim, name in self.v)
        self.args = Z.zero_block_norm_t(
            rows=rows, dim=dim, dtype16=self.kind, kind=Z.ZERO_NORM_LAYER if layer else Z.ZERO_NORM_RMS,
            norms=(Z.ZERO_NORM_POST if post else 0) | (Z.ZERO_NORM_PRE if pre else 0), rows_per_gate=gate_rows,
            eps=eps, residual_scale=scale,
            **{"ld_" + k: dim + pad for k in ("h", "x", "y", "z", "gate", "dy", "dz", "dx", "dh", "dgate")},
            **{k: a.data_ptr() for k, a in self.v.items()})

    def d(self, name):
        return self.v[name].double() if name in self.v else None

    def norm(self, a, w, b):
        c = a - a.mean(1, keepdim=True) if self.layer else a
        r = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + self.eps)
        hat = c * r
        return hat, r, hat * w + (b if b is not None else 0.0)

    def loss_of(self, a, hat, r):
        """What one fp32 rounding of a row's elements, or of its mean, may be in the normalised row."""
        lost = (a.abs() + a.abs().mean(1, keepdim=True)) * r if self.layer else hat.abs()
        return lost + hat.abs()

    def gates(self, gate):
        return gate.repeat_interleave(self.gate_rows, 0)[:self.rows] if gate is not None else 1.0

    def close(self, name, want, fp32):
        got = self.v[name].double()
        bound = fp32 * (1 + self.u16) + self.u16 * want.abs() + 2.0 ** -25
        bad = (got - want).abs() > bound
        assert not bool(bad.any()), (name, float(((got - want).abs() / bound).max()), int(bad.sum()))

    def run(self, back):
        outs = ["dx", "dh", "dgate"] + ["d" + k for k in VECTORS] if back else ["y", "z"]
        outs = [k for k in outs if getattr(self.args, k) and k in self.v]
        before = {k: storage(self.v[k]).clone() for k in self.v}
        s = torch.cuda.current_stream().cuda_stream
        if back:
            n = Z.zero_block_norm_workspace(self.args)
            ws = torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device="cuda")
            Z.zero_block_norm_backward(self.args, ws.data_ptr(), n, s)
        else:
            Z.zero_block_norm(self.args, s)
        for k, old in before.items():
            now = storage(self.v[k])
            if k in outs:
                mask = torch.ones_like(now, dtype=torch.bool)
                torch.as_strided(mask, self.v[k].shape, self.v[k].stride(), self.v[k].storage_offset()).fill_(False)
                now, old = now[mask], old[mask]
            assert torch.equal(now.view(torch.int16), old.view(torch.int16)), k

    def check_forward(self):
        self.run(False)
        h, x = self.d("h"), self.d("x") if "x" in self.v else 0.0
        u, lost = h, torch.zeros_like(h)
        if self.post:
            hat, r, u = self.norm(h, self.d("post_w"), self.d("post_b"))
            lost = 64 * U * (self.loss_of(h, hat, r) * self.d("post_w").abs() + u.abs())
        g = self.scale * self.gates(self.d("gate"))
        y = x + g * u
        lost_y = abs(g) * lost + 8 * U * (abs(x) + abs(g) * u.abs())
        self.close("y", y, lost_y)
        if self.pre:
            hat, r, z = self.norm(y, self.d("pre_w"), self.d("pre_b"))
            spread = lost_y * r + hat.abs() * (lost_y * r * hat.abs()).mean(1, keepdim=True)
            spread = spread + (lost_y * r).mean(1, keepdim=True) * self.layer
            self.close("z", z, (spread + 64 * U * self.loss_of(y, hat, r)) * self.d("pre_w").abs() + 8 * U * z.abs())

    def grads(self):
        """{output: (float64 gradient by the formula, bound of the fp32 part)}"""
        out = {}

        def through(a, w, dout, dout_err):
            hat, r, _ = self.norm(a, w, None)
            gw = dout * w
            core = gw - hat * (gw * hat).mean(1, keepdim=True)
            mag = gw.abs() + hat.abs() * (gw * hat).abs().mean(1, keepdim=True)
            e = dout_err * w.abs()
            err = e + hat.abs() * (e * hat.abs()).mean(1, keepdim=True)
            if self.layer:
                core = core - gw.mean(1, keepdim=True)
                mag = mag + gw.abs().mean(1, keepdim=True)
                err = err + e.mean(1, keepdim=True)
            rough = self.loss_of(a, hat, r)
            mag = mag + rough * (gw * hat).abs().mean(1, keepdim=True) + hat.abs() * (gw.abs() * rough).mean(1, keepdim=True)
            return r * core, r * (err + 256 * U * mag), hat, rough

        dx = self.d("dy") if self.args.dy else torch.zeros(self.rows, self.dim, dtype=torch.float64, device="cuda")
        err = torch.zeros_like(dx)
        n = self.rows + 64
        if self.pre:
            dz = self.d("dz")
            g, err, hat, rough = through(self.d("y"), self.d("pre_w"), dz, err)
            dx, err = dx + g, err + 4 * U * (dx.abs() + g.abs())
            out["dpre_w"] = ((dz * hat).sum(0, True), (n * U * (dz * hat).abs() + 64 * U * dz.abs() * rough).sum(0, True))
            out["dpre_b"] = (dz.sum(0, True), (n * U * dz.abs()).sum(0, True))
        out["dx"] = (dx, err)
        g = self.scale * self.gates(self.d("gate"))
        h = self.d("h")
        u, lost = h, torch.zeros_like(h)
        if self.post:
            hat, r, u = self.norm(h, self.d("post_w"), self.d("post_b"))
            lost = 64 * U * (self.loss_of(h, hat, r) * self.d("post_w").abs() + u.abs())
        if self.gate_rows:
            group = torch.arange(self.rows, device="cuda") // self.gate_rows
            terms = self.scale * dx * u
            e = abs(self.scale) * (err * (u.abs() + lost) + dx.abs() * lost) + (self.gate_rows + 64) * U * terms.abs()
            zero = torch.zeros_like(self.d("gate"))
            out["dgate"] = (zero.index_add(0, group, terms), zero.index_add(0, group, e))
        du, du_err = dx * g, err * abs(g) + 4 * U * (dx * g).abs()
        if self.post:
            dh, dh_err, hat, rough = through(h, self.d("post_w"), du, du_err)
            out["dh"] = (dh, dh_err)
            e = du_err * hat.abs() + n * U * (du * hat).abs() + 64 * U * du.abs() * rough
            out["dpost_w"] = ((du * hat).sum(0, True), e.sum(0, True))
            out["dpost_b"] = (du.sum(0, True), (du_err + n * U * du.abs()).sum(0, True))
        else:
            out["dh"] = (du, du_err)
        return out

    def check_backward(self):
        self.run(True)
        for name, (want, err) in self.grads().items():
            if name in self.v and getattr(self.args, name):
                self.close(name, want, err)


DIMS = [1, 2, 7, 8, 31, 64, 100, 255, 256, 257, 264, 768, 1000, 1023, 2048, 4096, 4100, 5000, 8191, 8192]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_dims(dim, layer, dtype):
    for rows, gate_rows in ((1, 1), (37, 5), (40, 40)):
        n = Norm(rows, dim, dtype, layer, gate_rows=gate_rows, seed=dim)
        n.check_forward()
        n.check_backward()


@pytest.mark.parametrize("rows", [1, 2, 9, 151, 153, 700, 2500, 5001])
@pytest.mark.parametrize("gate", [0, 1, 3, 7, 64, 700, "all"])
def test_rows_and_gate_groups(rows, gate):
    n = Norm(rows, 136, layer=True, gate_rows=rows if gate == "all" else gate, seed=rows)
    n.check_forward()
    n.check_backward()
    n = Norm(rows, 520, gate_rows=rows if gate == "all" else gate, seed=rows)
    n.check_backward()


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("gate_rows", [0, 1, 16])
def test_parts(post, pre, layer, bias, gate_rows):
    for x in (True, False):
        n = Norm(50, 320, layer=layer, post=post, pre=pre, bias=bias, gate_rows=gate_rows, x=x)
        n.check_forward()
        if not x:
            n.args.dy = None
        n.check_backward()


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (1, 0), (0, 1), (3, 5), (4, 4)])
def test_strides_and_starts(pad, shift):
    for dim in (264, 1001):
        n = Norm(33, dim, layer=True, gate_rows=4, pad=pad, shift=shift)
        n.check_forward()
        n.check_backward()


@pytest.mark.parametrize("mean", [30.0, 200.0])
def test_rows_with_a_large_mean(mean):
    n = Norm(20, 1024, "fp16", True, mean=mean)
    n.check_forward()
    n.check_backward()


@pytest.mark.parametrize("layer", [False, True])
def test_constant_and_zero_rows(layer):
    n = Norm(8, 512, "fp16", layer, eps=1e-6)
    n.v["h"][2] = 0.0
    n.v["h"][3] = 4.0
    n.v["y"][4] = 0.0
    n.v["y"][5] = -2.0
    n.check_backward()
    n.check_forward()


@pytest.mark.parametrize("which", ["dx", "dh", "dgate", "dpost_w", "dpre_b"])
def test_one_gradient_at_a_time(which):
    n = Norm(300, 264, layer=True, gate_rows=100)
    for name in ("dx", "dh", "dgate", "dpost_w", "dpost_b", "dpre_w", "dpre_b"):
        if name != which:
            setattr(n.args, name, None)
    n.check_backward()


def test_y_over_x_z_over_h_and_dx_over_dy():
    n = Norm(100, 264, layer=True, gate_rows=7)
    n.run(False)
    want_y, want_z = n.v["y"].clone(), n.v["z"].clone()
    keep_h, keep_x = n.v["h"].clone(), n.v["x"].clone()
    n.args.y, n.args.z = n.args.x, n.args.h
    Z.zero_block_norm(n.args, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(n.v["x"], want_y) and torch.equal(n.v["h"], want_z)
    n.v["h"].copy_(keep_h)
    n.v["x"].copy_(keep_x)
    n.args.y = n.v["y"].data_ptr()
    n.run(True)
    want = n.v["dx"].clone()
    n.args.dx = n.args.dy
    ws = torch.empty(Z.zero_block_norm_workspace(n.args), dtype=torch.uint8, device="cuda")
    Z.zero_block_norm_backward(n.args, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert torch.equal(n.v["dy"], want)


def test_no_rows():
    n = Norm(0, 64, layer=True)
    n.run(False)
    n.run(True)
    assert all(not bool(n.v["d" + k].any()) for k in VECTORS)


@pytest.mark.parametrize("layer", [False, True])
def test_gradients_are_the_differences(layer):
    """<gradient, direction> against central differences of the float64 forward."""
    n = Norm(12, 96, "fp16", layer, gate_rows=5, seed=8)

    def loss(v):
        u = n.norm(v["h"], v["post_w"], v.get("post_b"))[2]
        y = v["x"] + n.scale * n.gates(v["gate"]) * u
        z = n.norm(y, v["pre_w"], v.get("pre_b"))[2]
        return (y * dy).sum() + (z * dz).sum(), y

    dy, dz = n.d("dy"), n.d("dz")
    at = {k: n.d(k) for k in ("h", "x", "gate") + VECTORS if k in n.v}
    n.v["y"].copy_(loss(at)[1].to(n.t))
    n.run(True)
    for name in at:
        grad = n.d("d" + name)
        direction = grad.sign()
        value = [float(loss({**at, name: at[name] + s * direction})[0]) for s in (1e-6, -1e-6)]
        want, got = (value[0] - value[1]) / 2e-6, float((grad * direction).sum())
        # outputs' and y's roundings of 2^-11, y's amplified by the pre-norm's second derivative
        # (|dz| |z| / std^2, below 4 here), all of one sign at worst
        assert abs(got - want) <= 2.0 ** -8 * abs(want), (name, got, want)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_values_that_are_not_finite_stay_in_their_rows(bad):
    n = Norm(40, 264, layer=True, gate_rows=0)
    n.v["h"][7, 100] = bad
    n.run(False)
    rows = ~torch.isfinite(n.v["z"].float()).all(1)
    assert rows.nonzero().flatten().tolist() == [7]


def test_another_stream_and_a_graph():
    n = Norm(300, 520, layer=True, gate_rows=100)
    n.run(False)
    n.run(True)
    outs = [k for k in n.v if k in ("y", "z", "dx", "dh", "dgate") or k[1:] in VECTORS]
    n.run(True)
    want = {k: n.v[k].clone() for k in outs}
    ws = torch.empty(Z.zero_block_norm_workspace(n.args), dtype=torch.uint8, device="cuda")
    for k in ("z", "dx", "dh", "dgate"):
        n.v[k].zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        Z.zero_block_norm(n.args, side.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_block_norm_backward(n.args, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    graph.replay()
    torch.cuda.synchronize()
    for k in outs:
        assert torch.equal(n.v[k], want[k]), k
