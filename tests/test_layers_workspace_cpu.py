"""Workspace sizes of the layer operators: a call asks for what its split
partials take and no more. Host only."""

from __future__ import annotations

import pytest

from block_scaled_fp8_linear_amd import _lib as L

OPS = ("linear_act", "linear_act_backward", "glu", "glu_backward")
COLUMNS = {"linear_act": lambda n, k: n, "linear_act_backward": lambda n, k: k,
           "glu": lambda n, k: 2 * n, "glu_backward": lambda n, k: k}


def outputs(op, m, n, k):
    """fp32 bytes of one set of partials over all of a product's columns."""
    return 4 * m * COLUMNS[op](n, k)


# Products a little larger than whole rounds of the chip: only the tile columns
# left over are split. `columns` is how many those are, at most: what lies past
# the last whole round of 256 tiles (256 x 256, the pair's 256 x 128).
LEFT_OVER = [
    ("glu", 6144, 13824, 5120, 2 * 384), ("linear_act", 6144, 27648, 5120, 768),
    ("linear_act", 8192, 12544, 4096, 256), ("glu_backward", 4096, 12800, 5120, 1024),
    ("linear_act", 2048, 8448, 4096, 256), ("linear_act_backward", 2048, 4096, 8448, 256),
    ("glu", 4096, 24704, 25216, 2 * 128),
]


@pytest.mark.parametrize("op,m,n,k,columns", LEFT_OVER, ids=lambda v: str(v))
def test_columns_left_over(op, m, n, k, columns):
    """At most 32 splits of the columns that are split."""
    need = L.layer_workspace_size(op, m, n, k)
    assert 0 < need <= 32 * 4 * m * columns + 256
    # and, as every such rest, less than the chip's 256 tiles in 32 splits each
    assert need < outputs(op, m, n, k)


def test_workspace_stays_near_what_the_chip_holds():
    """Splits are there to give every CU a tile, so partials of a few rounds of
    256 tiles of 256 x 256 are enough: none of these sizes asks for more than
    eight rounds, beside the padded gradients and column sums of the backward
    passes."""
    round_bytes = 256 * 256 * 256 * 4
    for op in OPS:
        for m in (1, 16, 33, 300, 512, 2048, 4096, 6144, 8192, 65536):
            for n in (8, 1003, 4096, 8448, 13824, 24704, 25600):
                for k in (16, 656, 5120, 8448, 25216):
                    need = L.layer_workspace_size(op, m, n, k)
                    products = {"linear_act": 0, "linear_act_backward": 1, "glu": 0, "glu_backward": 2}[op]
                    pads = products * 2 * m * (n + 7) if n % 8 else 0
                    sums = 256 * n * 4 if op == "linear_act_backward" else 0
                    assert need <= 8 * round_bytes + pads + sums + 1024, (op, m, n, k, need)
