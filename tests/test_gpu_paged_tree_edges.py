"""Trees of drafted tokens over a paged cache: workspaces of the size that the library names, in every kernel,
and maps beside corrupt row bounds."""
import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa
from oracle import paged
from test_gpu_paged import _errors, _i32
from test_gpu_paged_tree import T5D, Tree, _parents

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    _errors()


# Contexts that every kernel cuts (beyond 1024 keys), so that partial rows are written: up to 16 rows a key/value
# head, up to 64, up to 128, more of them, blocks of 128 rows that fill the SMs, and requests of all kinds.
WORKSPACES = {
    "few": dict(lq=[5, 3, 1], ctx=[1900, 700, 4000], hq=6, hkv=2, d=64),
    "few_d128": dict(lq=[4, 3, 0, 2], ctx=[5000, 130, 7, 1800], hq=8, hkv=2, d=128),
    "rows64": dict(lq=[30, 17], ctx=[6000, 1500], hq=4, hkv=2, d=64),
    "rows64_d128": dict(lq=[15, 9], ctx=[1100, 7000], hq=8, hkv=2, d=128),
    "rows128": dict(lq=[60, 100], ctx=[1400, 3000], hq=2, hkv=2, d=64),
    "rows128_d128": dict(lq=[31, 20], ctx=[5000, 1200], hq=8, hkv=2, d=128),
    "blocks": dict(lq=[140, 30], ctx=[3000, 2000], hq=2, hkv=2, d=64),
    "blocks_d128": dict(lq=[61, 90], ctx=[2500, 1300], hq=8, hkv=2, d=128),
    "tile": dict(lq=[140] * 12, ctx=[1100 + 40 * i for i in range(12)], hq=8, hkv=8, d=64),
    "tile_d128": dict(lq=[80] * 13, ctx=[1100 + 40 * i for i in range(13)], hq=16, hkv=8, d=128),
    "mixed": dict(lq=[1, 60, 3, 0, 16, 40], ctx=[2000, 30, 1000, 5, 800, 4000], hq=8, hkv=2, d=64),
}


@pytest.mark.parametrize("name", WORKSPACES)
def test_nothing_behind_the_workspace(name):
    t = Tree(seed=len(name), page=64, t5=T5D, **WORKSPACES[name])
    p = t.p
    k = int(max(p.lk))
    size = fa.fat_paged_attn_workspace_size(p.q, p.kc, _i32(p.cu), t.most, k)
    assert size > 0
    first = None
    for fill in (0xff, 0x7f):
        buf = torch.full((size + 4096,), fill, dtype=torch.uint8, device=DEV)
        out, lse = t.run(workspace=buf[:size])
        assert _errors() == 0
        assert (buf[size:] == fill).all() and not (buf[:size] == fill).all()
        if first is None:
            t.check(out, lse)
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    if p.total != p.n * t.most:  # (else the few-row kernel, whose rows are counted, is not launched)
        with pytest.raises(fa.FatAttnError):
            t.run(workspace=buf[:size - 1])
    with pytest.raises(fa.FatAttnError):
        t.run(workspace=buf[:1024])
    assert _errors() == 0


# cu_seqlens_q with one bad entry, and the requests whose rows no other request claims: theirs are right; rows of
# a request with bounds outside the arrays or out of order stay as they were, unless another one claims them.
@pytest.mark.parametrize("at,value,right,left", [
    (1, -3, (2, 3), (0, 13)), (2, 1000, (0, 3), (9, 33)), (2, 3, (3,), (0, 0)), (4, 1000, (0, 1, 2), (33, 39)),
    (4, 30, (0, 1), (0, 0)), (2, 9, (0, 3), (0, 0)), (0, 5, (1, 2, 3), (0, 5))])
def test_plan_beside_corrupt_bounds(at, value, right, left):
    rng = np.random.default_rng(4)
    lq, most, words = [9, 4, 20, 6], 20, 2
    lk = np.array(lq) + 10
    par = _parents(rng, lq, 3)
    cu = np.concatenate([[0], np.cumsum(lq)])
    pos, mask = paged.tree_plan(par, cu, lk, 39, most, words)
    bad = cu.copy()
    bad[at] = value
    guard = 64
    p = torch.full((39 + 2 * guard,), -9, dtype=torch.int32, device=DEV)
    m = torch.full((39 + 2 * guard, words), -9, dtype=torch.int32, device=DEV)
    fa.fat_paged_tree_plan(_i32(par), _i32(bad), _i32(lk), most, positions=p[guard:-guard],
                           tree_mask=m[guard:-guard])
    # (bounds that are still in order only make another request, whose parents are those of other nodes)
    assert _errors() & (fa.FAT_DEVERR_INDEX if at == 0 else fa.FAT_DEVERR_SEQLENS)
    p, m = p.cpu().numpy(), m.cpu().numpy()
    for x in (p, m):
        assert (x[:guard] == -9).all() and (x[-guard:] == -9).all()
    p, m = p[guard:-guard], m[guard:-guard]
    for i in right:
        rows = slice(cu[i], cu[i + 1])
        np.testing.assert_array_equal(p[rows], pos[rows])
        np.testing.assert_array_equal(m[rows], mask[rows])
    assert (p[slice(*left)] == -9).all() and (m[slice(*left)] == -9).all()
