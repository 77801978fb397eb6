"""The output layer's cross-entropy without a GPU: what the host decides before a launch."""
import ctypes

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


@pytest.mark.parametrize("pairs", [1, 5, 74, 76, 128])
@pytest.mark.parametrize("vocab,dim", [(1, 8), (300, 72), (5000, 40), (32003, 776), (32768, 1024),
                                       (131072, 2048), (700001, 264), (1100000, 64), (2000, 16384)])
@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_does_for_fewer_rows(lib, pairs, vocab, dim, backward):
    """A workspace made for a number of rows holds every call of fewer."""
    rows = sorted({*range(1, 300, 7), *range(256, 6000, 64), *(256 * i + o for i in range(1, 140) for o in (0, 1)),
                   128, 129, 1535, 1536, 1537, 50000, 100000, 262144})
    used, before = ctypes.c_size_t(), 0
    for n in rows:
        size = lib.fat_attn_debug_head_workspace(_shape(n, vocab, dim), pairs, backward, ctypes.byref(used))
        assert used.value <= size and size >= before, (n, used.value, size, before)
        before = size
