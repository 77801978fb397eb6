"""Trees of drafted tokens over a paged cache: workspaces of the size that the library names, in every kernel."""
import pytest
import torch

import attention_relative_position_gb300 as fa
from test_gpu_paged import _errors, _i32
from test_gpu_paged_tree import T5D, Tree

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
