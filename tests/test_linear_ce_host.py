"""The output layer's cross-entropy without a GPU: what the host decides before a launch."""
import pytest

import attention_relative_position_gb300 as fa
from attention_relative_position_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def _shape(rows, vocab, dim):
    return fa._LinearCeShape(rows, vocab, dim, dim, dim, 1.0, 0.0, None)


@pytest.mark.parametrize("pairs", [1, 2, 7, 74, 75, 76])
@pytest.mark.parametrize("dim", [8, 512, 776, 2048])
def test_columns_of_a_product(lib, pairs, dim):
    """A product on a pair of SMs with 256 rows has a multiple of 32 columns, 256 at most."""
    rows = list(range(1, 600)) + [700, 1025, 1536, 2077, 8192, 16384, 50000]
    for n in rows:
        for vocab in (1, 17, 300, 3001, 5000, 32003, 50021, 131072):
            cols = lib.fat_attn_debug_head_columns(_shape(n, vocab, dim), pairs)
            assert cols % 32 == 0 and 32 <= cols <= 256, (n, vocab, cols)
            assert n > 128 or cols >= n, (n, cols)
    assert lib.fat_attn_debug_head_columns(_shape(0, 5, dim), pairs) == 0
    assert lib.fat_attn_debug_head_columns(_shape(4, 0, dim), pairs) == 0
