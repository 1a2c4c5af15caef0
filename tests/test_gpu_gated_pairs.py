"""zero_gated_backward at sizes whose gradients are made by pairs of SMs (tiles of 256 x 256), against float64; bounds as in
test_gpu_gated.py.  Whole tiles of both kinds, dx in parts of its inner dimension, the weights' gradients in parts, rows on
the 16-byte grid and off it, and any of the gradients alone."""
import pytest
import torch
from test_gpu_gated import Block, call

import zero_sharded_mixed_03_gb300 as Z

pytestmark = pytest.mark.gpu
# few rows and many tiles; many rows; the weights' gradients in parts; dx in parts; odd in every size
SIZES = [(140, 4096, 4900), (1500, 2000, 2500), (4096, 512, 1024), (1100, 1000, 3000), (1001, 2003, 2501)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_backward(m, k, n, layout):
    for dtype, act, pad, accumulate in (("bf16", "silu", 0, False), ("fp16", "gelu_tanh", 0, True), ("bf16", "relu", 8, True),
                                        ("bf16", "gelu", 3, False)):
        Block(m, k, n, dtype, layout, act, pad=pad, seed=m + pad).check_backward(accumulate=accumulate)


@pytest.mark.parametrize("layout", ["out_in", "in_out"])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_whole_numbers_are_exact(m, k, n, layout):
    """dg and du are whole numbers of at most 4, every sum below 2^24."""
    for act in ("none", "relu"):
        Block(m, k, n, "bf16", layout, act, whole=True, seed=k).check_backward(exact=True)


@pytest.mark.parametrize("wanted", [("dx",), ("dw_gate",), ("dw_up", "db_gate"), ("dw_gate", "dw_up"), ("dx", "dw_up"),
                                    ("dx", "db_gate", "db_up")])
def test_some_gradients_only(wanted):
    for m, k, n in SIZES[1:4]:
        b = Block(m, k, n, seed=1)
        for name in ("dx", "dw_gate", "dw_up", "db_gate", "db_up"):
            if name not in wanted:
                setattr(b.args, name, None)
        b.check_backward()


@pytest.mark.parametrize("m,k,n", SIZES[2:])
def test_repeats_streams_and_graphs(m, k, n):
    names = ("dx", "dw_gate", "dw_up", "db_gate", "db_up")
    b = Block(m, k, n, "bf16", "in_out", pad=8, seed=2)
    call(b.args, True)
    torch.cuda.synchronize()
    want = {v: getattr(b, v).clone() for v in names}

    def same():
        torch.cuda.synchronize()
        assert all(torch.equal(want[v], getattr(b, v)) for v in names)
        for v in names:
            getattr(b, v).zero_()
        torch.cuda.synchronize()

    same()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ws = call(b.args, True, side)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Z.zero_gated_backward(b.args, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    for _ in range(2):
        graph.replay()
        same()
