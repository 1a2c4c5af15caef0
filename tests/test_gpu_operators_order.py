"""Calls of zero_linear_backward back to back on one workspace, whose inputs other kernels rewrite between them.

Whole numbers whose sums stay below 2^24 have one answer, so every call of a long loop, and of a replayed
graph, is compared with its inputs' float64 products element by element.
"""
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
# small ones, of which several run at one time; rows off the 16-byte grid; more tiles than run at one time
SHAPES = [(16, 64, 128), (200, 320, 448), (77, 101, 163), (129, 65, 257), (64, 4096, 64), (1536, 1088, 2560)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


class Calls:
    """Sets of inputs, one set of buffers that the calls read and add to, and what each call leaves."""

    def __init__(self, shape, layout, act, sets=3):
        m, k, n = shape
        gen = torch.Generator().manual_seed(sum(shape))

        def whole(r, c, hi=2):
            return torch.randint(-hi, hi + 1, (r, c), generator=gen).to(torch.bfloat16).cuda()

        w_shape = (n, k) if layout == Z.ZERO_WEIGHT_OUT_IN else (k, n)
        self.inputs = [dict(x=whole(m, k), w=whole(*w_shape), pre=whole(m, n), dy=whole(m, n), dw=whole(*w_shape),
                            dbias=whole(1, n)) for _ in range(sets)]
        self.want = []
        for s in self.inputs:
            dz = s["dy"].double() * ((s["pre"] > 0).double() if act else 1.0)
            w = s["w"].double() if layout == Z.ZERO_WEIGHT_OUT_IN else s["w"].double().t()
            dw = dz.t() @ s["x"].double() if layout == Z.ZERO_WEIGHT_OUT_IN else s["x"].double().t() @ dz
            self.want.append([t.to(torch.bfloat16) for t in (dz @ w, dw + s["dw"].double(),
                                                            dz.sum(0, keepdim=True) + s["dbias"].double())])
        self.buf = {k: torch.empty_like(v) for k, v in self.inputs[0].items()}
        self.buf["dx"] = torch.empty_like(self.buf["x"])
        self.args = Z.zero_linear_t(rows=m, in_features=k, out_features=n, dtype16=Z.ZERO_BF16, layout=layout,
                                    activation=Z.ZERO_ACT_RELU if act else Z.ZERO_ACT_NONE, flags=Z.ZERO_LINEAR_ACCUMULATE,
                                    **{k: v.data_ptr() for k, v in self.buf.items()})
        self.bytes = Z.zero_linear_workspace(self.args, True)
        self.ws = torch.full((max(16, self.bytes),), 0xFF, dtype=torch.uint8, device="cuda")
        self.wrong = torch.zeros(3, dtype=torch.int64, device="cuda")

    def call(self, i):
        for k, v in self.inputs[i].items():
            self.buf[k].copy_(v)
        Z.zero_linear_backward(self.args, self.ws.data_ptr(), self.bytes, torch.cuda.current_stream().cuda_stream)
        for j, (name, want) in enumerate(zip(("dx", "dw", "dbias"), self.want[i])):
            self.wrong[j] += (self.buf[name] != want).sum()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("layout", [Z.ZERO_WEIGHT_OUT_IN, Z.ZERO_WEIGHT_IN_OUT])
@pytest.mark.parametrize("act", [False, True])
def test_gradients_in_a_loop_and_in_a_graph(shape, layout, act):
    calls = Calls(shape, layout, act)
    for i in range(30):
        calls.call(i % 3)
    assert calls.wrong.tolist() == [0, 0, 0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(6):
            calls.call(i % 3)
    for _ in range(100):
        graph.replay()
    torch.cuda.synchronize()
    assert calls.wrong.tolist() == [0, 0, 0]


@pytest.mark.parametrize("only", ["dx", "dw", "dbias"])
def test_one_gradient_alone(only):
    calls = Calls((200, 320, 448), Z.ZERO_WEIGHT_OUT_IN, True)
    for name in ("dx", "dw", "dbias"):
        if name != only:
            setattr(calls.args, name, None)
    at = ("dx", "dw", "dbias").index(only)
    calls.bytes = Z.zero_linear_workspace(calls.args, True)
    for i in range(30):
        calls.call(i % 3)
    assert int(calls.wrong[at]) == 0


def test_weights_written_by_the_launch_before():
    """One optimizer step writes the 16-bit gains that the next launch, a norm, reads: 400 times over, against
    the same with a wait between them."""
    dim, rows = 2048, 700
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(rows, dim, generator=gen, device="cuda").to(torch.bfloat16)
    outs = []
    for wait in (False, True):
        p = torch.ones(dim, device="cuda")
        p16 = p.to(torch.bfloat16)
        g = torch.randn(dim, generator=torch.Generator().manual_seed(2)).cuda()
        z = torch.empty_like(h)
        total = torch.zeros(rows, dim, device="cuda")
        opt = Z.zero_adamw_create([dim], 32, Z.ZERO_BF16, Z.ZERO_FP32)
        info = Z.zero_adamw_info(opt)
        m, v, ws = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in
                    (info.moment_bytes, info.moment_bytes, info.workspace_bytes))
        s = torch.cuda.current_stream().cuda_stream
        Z.zero_adamw_bind(opt, [p.data_ptr()], [p16.data_ptr()], [g.data_ptr()], m.data_ptr(), v.data_ptr(), None,
                          ws.data_ptr(), 0, s)
        args = Z.zero_block_norm_t(rows=rows, dim=dim, dtype16=Z.ZERO_BF16, kind=Z.ZERO_NORM_RMS, norms=Z.ZERO_NORM_PRE,
                                   eps=1e-5, residual_scale=1.0, h=h.data_ptr(), pre_w=p16.data_ptr(), z=z.data_ptr())
        try:
            for _ in range(400):
                Z.zero_adamw_step(opt, Z.hyper(lr=0.05), 1.0, s)
                if wait:
                    torch.cuda.synchronize()
                Z.zero_block_norm(args, s)
                total += z
            torch.cuda.synchronize()
        finally:
            Z.zero_adamw_destroy(opt)
        outs.append(total)
    assert torch.equal(*outs)
