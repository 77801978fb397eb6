"""GPU parity of the output layer's cross-entropy at the edges of its tiles and workspaces, against fp64."""
import pytest
import torch

import attention_relative_position_gb300 as fa
from test_gpu_linear_ce import _check_bwd, _check_fwd, _errors, _inputs

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


# fewer rows may be cut into more tiles, pieces or splits than the rows that the workspace was made for
@pytest.mark.parametrize("rows,more,vocab,dim", [
    (256, 257, 5000, 64), (128, 129, 40000, 64), (500, 1537, 9000, 72), (1024, 1280, 131072, 64),
    (300, 16385, 5000, 136), (512, 900, 20000, 1032)])
def test_workspace_of_more_rows(rows, more, vocab, dim):
    h, w, t = _inputs(rows, vocab, dim, ignored=0.1)
    size = [fa.fat_linear_cross_entropy_workspace_size(more, vocab, dim, backward=b) for b in (False, True)]
    ws = [torch.full((n + 4096,), 0xff, dtype=torch.uint8, device="cuda") for n in size]
    _check_fwd(h, w, t, workspace=ws[0][:-4096])
    _check_bwd(h, w, t, grad_scale=1.0 / rows, workspace=ws[1][:-4096])
    assert all((x[-4096:] == 0xff).all() for x in ws)
