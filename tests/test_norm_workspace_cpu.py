"""Sizes of layer norm's workspace."""
import pytest

from linear_token_mixer_gb300 import build as B_
from linear_token_mixer_gb300 import fw


@pytest.fixture(scope="module")
def L():
    B_.build()
    return fw.lib()


@pytest.mark.parametrize("rows,width", [(1, 20000), (1000, 20000), (100000, 2 ** 17), (700, 2 ** 20),
                                        (5, 2 ** 24), (100, 2 ** 24)])
def test_wide_rows_keep_few_partial_rows(L, rows, width):
    """Rows wider than a block's registers: at most 608 blocks of 256 columns sum them, and each block
    writes its columns' part of two rows (a partial row of dweight and one of dbias)."""
    blocks = (width + 255) // 256
    most = max(1, min(rows, 608 // blocks))
    assert 0 < L.fw_layer_norm_workspace(rows, width) <= most * 2 * width * 4
