"""zero_block_norm with many wide rows: those that come through shared memory (RowPipe).

Rows are staged where all threads of a block hold as much of a row, a row takes more than a warp and
there are more rows than blocks that run at one time, so that the ring of stages wraps in every block.
Tolerances are test_gpu_block_norm.py's.
"""
import pytest
import torch

import zero_sharded_mixed_03_gb300 as Z
from test_gpu_block_norm import Norm, VECTORS

pytestmark = pytest.mark.gpu
# eight, sixteen and thirty-two elements a thread forward, eight and sixteen backward
WIDE = [(768, 9000), (1280, 6000), (2048, 5000), (2560, 2500), (4096, 2500)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    Z.lib()
    yield
    Z.zero_operators_check()


@pytest.mark.parametrize("dim,rows", WIDE)
@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate_rows", [0, 1, 7, "all"])
def test_many_wide_rows(dim, rows, layer, gate_rows):
    n = Norm(rows, dim, "fp16" if dim == 1280 else "bf16", layer, gate_rows=rows if gate_rows == "all" else gate_rows, seed=dim)
    n.check_forward()
    n.check_backward()


@pytest.mark.parametrize("gate_rows", [0, 1, 1300])
@pytest.mark.parametrize("layer", [False, True])
def test_the_widest_rows(gate_rows, layer):
    n = Norm(1300, 8192, layer=layer, gate_rows=gate_rows, seed=4)
    n.check_forward()
    n.check_backward()


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate_rows", [0, 1, 64])
@pytest.mark.parametrize("post,pre,x", [(True, True, False), (True, False, True), (False, True, True), (True, False, False),
                                        (False, True, False)])
def test_parts_of_many_wide_rows(layer, gate_rows, post, pre, x):
    """Tensors that are not there read as zeros from their places in a stage."""
    for dim, rows in ((768, 7000), (2048, 2600)):
        n = Norm(rows, dim, layer=layer, post=post, pre=pre, gate_rows=gate_rows, x=x, seed=dim)
        n.check_forward()
        if not x:
            n.args.dy = None
        n.check_backward()


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("rows", [609, 760, 761, 1217, 1520, 1521])
def test_rows_around_a_whole_number_of_rounds(layer, rows):
    n = Norm(rows, 2048, layer=layer, gate_rows=1, seed=rows)
    n.check_forward()
    n.check_backward()


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("gate_rows", [1, 100])
def test_in_place(layer, gate_rows):
    """y over x, z over h and dx over dy give what separate buffers do."""
    for dim, rows in ((768, 7000), (4096, 1500)):
        n = Norm(rows, dim, layer=layer, gate_rows=gate_rows, seed=dim)
        n.run(False)
        n.run(True)
        want = {k: n.v[k].clone() for k in ("y", "z", "dx", "dh", "dgate") + tuple("d" + k for k in VECTORS if k in n.v)}
        for k in ("dh", "dgate"):
            n.v[k].zero_()
        stream = torch.cuda.current_stream().cuda_stream
        n.args.dx = n.args.dy
        ws = torch.empty(Z.zero_block_norm_workspace(n.args), dtype=torch.uint8, device="cuda")
        Z.zero_block_norm_backward(n.args, ws.data_ptr(), ws.numel(), stream)
        n.args.y, n.args.z = n.args.x, n.args.h
        Z.zero_block_norm(n.args, stream)
        for k, w in want.items():
            assert torch.equal(n.v[{"y": "x", "z": "h", "dx": "dy"}.get(k, k)], w), k


def test_padded_strides():
    n = Norm(3000, 1280, layer=True, gate_rows=1, pad=8, shift=8)
    n.check_forward()
    n.check_backward()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_values_that_are_not_finite_stay_in_their_rows(bad):
    n = Norm(5000, 2048, gate_rows=1)
    n.v["h"][77, 100] = bad
    n.v["h"][4999, 2047] = bad
    n.run(False)
    rows = ~torch.isfinite(n.v["z"].float()).all(1)
    assert rows.nonzero().flatten().tolist() == [77, 4999]


@pytest.mark.parametrize("rows_per_gate", [301, 1 << 60, (1 << 63) - 1])
@pytest.mark.parametrize("layer", [False, True])
def test_a_gate_row_for_more_rows_than_there_are(rows_per_gate, layer):
    for rows, dim in ((1, 136), (300, 136), (300, 2048)):
        n = Norm(rows, dim, layer=layer, gate_rows=rows)
        n.args.rows_per_gate = rows_per_gate
        n.check_forward()
        n.check_backward()
