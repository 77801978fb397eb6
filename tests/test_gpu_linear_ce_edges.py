"""GPU parity of the output layer's cross-entropy at the edges of its tiles and workspaces, against fp64."""
import pytest

from test_gpu_linear_ce import _check_fwd, _errors, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    _errors()


# every width of a product: up to 128 rows they are the columns, above it vocabulary entries (70 tiles of
# that many fit a GPU of 70 to 76 pairs in one round)
@pytest.mark.parametrize("rows", [1, 15, 16, 31, 32, 33, 48, 63, 65, 80, 95, 97, 112, 127])
def test_widths_of_few_rows(rows):
    h, w, t = _inputs(rows, 700, 72, ignored=0.2 if rows > 2 else 0.0)
    _check_fwd(h, w, t)


@pytest.mark.parametrize("dim", [72, 1032])
@pytest.mark.parametrize("cols", range(32, 257, 32))
def test_widths_of_many_rows(cols, dim):
    h, w, t = _inputs(200, 70 * cols - 5, dim, ignored=0.2)
    _check_fwd(h, w, t)
