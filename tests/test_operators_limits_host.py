"""Sizes at the ends of the operators' ranges, on the host alone."""
import pytest

import zero_sharded_mixed_03_gb300 as Z


def norm(rows, dim, rows_per_gate, layer):
    return Z.zero_block_norm_t(rows=rows, dim=dim, dtype16=Z.ZERO_BF16, kind=Z.ZERO_NORM_LAYER if layer else Z.ZERO_NORM_RMS,
                               norms=Z.ZERO_NORM_PRE | Z.ZERO_NORM_POST, rows_per_gate=rows_per_gate, eps=1e-5,
                               residual_scale=1.0, h=4096, gate=8192, y=16384, dy=32768, dz=65536, dx=4096 * 99, dh=4096 * 100,
                               dgate=4096 * 101, dpost_w=4096 * 102, dpre_w=4096 * 103)


@pytest.mark.parametrize("rows_per_gate", [5001, 1 << 59, (1 << 60) + 1, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("rows,dim", [(1, 64), (40, 136), (5000, 136), (5000, 8192)])
@pytest.mark.parametrize("layer", [False, True])
def test_a_gate_row_for_more_rows_than_there_are(rows_per_gate, rows, dim, layer):
    """One for all of them, whatever the number: the same cut and the same workspace."""
    assert Z.zero_block_norm_workspace(norm(rows, dim, rows_per_gate, layer)) == Z.zero_block_norm_workspace(norm(rows, dim, rows, layer))
