"""Rows at the end of what one launch holds (CPU only): refused before anything
is enqueued, by the threads that the kernels really take."""
import pytest

from gated_deltanet_chunked_rule_amd import layer
from test_layer_refusals import last


# lanes a row as the launcher has them: powers of two up to 2048 values, whole waves of one or two vectors behind
LANES = [(1, 16), (128, 16), (129, 32), (300, 64), (1024, 128), (2048, 256), (2049, 192), (4096, 256), (4097, 576), (4608, 576),
         (5120, 640), (5121, 704), (6144, 768), (6145, 448), (8192, 512), (8193, 576), (16384, 1024)]


@pytest.mark.parametrize("dim,lanes", LANES)
def test_block_norm_refuses_rows_beyond_a_launch(dim, lanes):
    size = layer._entry("gdr_block_norm_bwd_workspace_size")
    most = (2 ** 32 - 1) // lanes
    for rows in (most + 1, 2 ** 62, 2 ** 63 - 1):
        assert size(layer._BlockNormShape(rows, dim, 0, 1e-6, 0, 0, 0)) == 0 and "too many rows" in last(), rows
    for rows in (most - 256, 1):                # a workgroup's rows and 256 threads less than 2^32
        assert size(layer._BlockNormShape(rows, dim, 0, 1e-6, 0, 0, 0)) > 0, rows
