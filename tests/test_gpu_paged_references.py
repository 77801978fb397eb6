"""Attention over a paged cache beside biases that mask with large finite numbers: what such keys leave in a
row's running maximum must not reach the row's other keys. Trees of drafted tokens against the fp64 oracle."""
import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa  # noqa: F401
from test_gpu_paged import _errors, _wide
from test_gpu_paged_tree import T5D, Tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_error_word():
    _errors()


def _patterns(p, low, pattern, rng):
    """Buckets of heads that mask: every near one (whole tiles of masked keys come first), every second
    distance, or any."""
    b = p.bias  # [32, heads]: distances 0 to 15, then up to 128
    hide = np.zeros(b.shape, bool)
    if pattern == "near":
        hide[:31] = True
    elif pattern == "odd":
        hide[1:16:2, ::2] = True
        hide[0:16:2, 1::2] = True
        hide[16:28] = True
    else:
        hide = rng.random(b.shape) < 0.7
        hide[31, ::2] = False
    b[torch.as_tensor(hide, device=b.device)] = low
    return hide


# A masked key's weight beside any other key of its row is exp(-1e6 + logits) = 0 in any arithmetic, so the
# oracle leaves those keys out. A row that sees nothing else has logits that fp32 rounds to within 2^-24 of the
# bias: its lse is the bias, up to some such roundings, a logit and the logarithm of the number of keys, and its
# output a mean of values.
def _check(t, out, lse, low):
    p = t.p
    b = p.bias.cpu().numpy()
    p.bias[p.bias <= low] = -float("inf")
    ro, rl, a, s, _ = t.oracle()
    big = float(np.abs(b[b > low]).max(initial=0.0))
    ex = (p.d * s + 4 * (s + big)) * 2.0 ** -24
    got, gl = _wide(out[:p.total]), lse.cpu().numpy()[:, :p.total].astype(np.float64)
    assert np.isfinite(got).all() and np.isfinite(gl).all()
    fin = np.isfinite(rl)
    assert (np.abs(gl[~fin] - low) <= 2.0 ** -21 * abs(low) + s + 9).all()
    most = np.nanmax(np.abs(_wide(p.vc)))  # (places behind the last keys hold NaN)
    assert (np.abs(got) <= most * (1 + 2.0 ** -7)).all()
    assert fin.mean() > 0.2
    err, tol = np.abs(got - ro), 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ex + 2.0 ** -18) * a * 1.01 + 1e-30
    rows = fin.T
    assert (err[rows] <= tol[rows]).all(), (err[rows] / tol[rows]).max()
    ltol = ex + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl[fin])
    assert (np.abs(gl[fin] - rl[fin]) <= ltol).all(), np.abs(gl[fin] - rl[fin]).max()


ITEMS = {
    "few": dict(lq=[5, 3], ctx=[1500, 140], hq=2, hkv=2, d=64),
    "rows64": dict(lq=[30, 25], ctx=[1500, 133], hq=2, hkv=2, d=64),
    "rows64_d128": dict(lq=[12, 15], ctx=[700, 2300], hq=8, hkv=2, d=128),
    "rows128": dict(lq=[60, 100], ctx=[300, 1400], hq=2, hkv=2, d=64),
    "rows128_d128": dict(lq=[61, 24], ctx=[1300, 300], hq=8, hkv=2, d=128),
    "tile": dict(lq=[140] * 12, ctx=[400] * 12, hq=8, hkv=8, d=64),
}


@pytest.mark.parametrize("low", [-1e6, -1e10, -1e30, -2e38])
@pytest.mark.parametrize("std", [1.0, 12.0])
@pytest.mark.parametrize("pattern", ["near", "odd", "any"])
@pytest.mark.parametrize("item", ITEMS)
def test_large_masking_biases(item, pattern, std, low):
    t = Tree(page=64, t5=T5D, std=std, seed=5, **ITEMS[item])
    _patterns(t.p, low, pattern, np.random.default_rng(9))
    out, lse = t.run()
    assert _errors() == 0
    _check(t, out, lse, low)


# The tile kernel: trees that fill the GPU with blocks of 128 rows, and chains (fat_paged_attn), whose keys are
# a tree's of one path.
CHAINS = {
    "few": dict(lq=[5, 3], ctx=[1500, 140], hq=2, hkv=2, d=64),
    "few_d128": dict(lq=[4, 2], ctx=[700, 2300], hq=8, hkv=2, d=128),
    "tile": dict(lq=[300, 25], ctx=[900, 133], hq=2, hkv=2, d=64),
    "tile_d128": dict(lq=[130, 40, 17], ctx=[700, 0, 2300], hq=4, hkv=2, d=128),
}


@pytest.mark.parametrize("low", [-1e6, -1e10, -1e30, -2e38])
@pytest.mark.parametrize("std", [1.0, 12.0])
@pytest.mark.parametrize("pattern", ["near", "odd", "any"])
@pytest.mark.parametrize("chain", [None, *CHAINS])
def test_large_masking_biases_of_tiles(chain, pattern, std, low):
    case = CHAINS[chain] if chain else dict(lq=[140] * 12, ctx=[400] * 12, hq=8, hkv=8, d=128)
    t = Tree(page=64, t5=T5D, std=std, seed=6, reach=1 if chain else 3, **case)
    _patterns(t.p, low, pattern, np.random.default_rng(8))
    if chain:
        t.p.causal = True
        out, lse = t.p.run()
    else:
        out, lse = t.run()
    assert _errors() == 0
    _check(t, out, lse, low)


# Far keys that are masked, in items of which a part begins behind the near ones; then all keys, whose rows' logits
# differ by hundreds: beside such biases fp32 cannot tell the keys apart, but every row has a result.
@pytest.mark.parametrize("low", [-1e9, -1e30, 1e10])
@pytest.mark.parametrize("std", [1.0, 12.0])
@pytest.mark.parametrize("lq,hq,hkv,d", [([30], 2, 2, 64), ([30], 4, 2, 128), ([100], 1, 1, 64), ([70], 1, 1, 128),
                                         ([5], 2, 2, 64), ([16] * 3, 4, 2, 128)])
def test_masked_far_keys_in_parts(lq, hq, hkv, d, std, low):
    t = Tree(lq, [6000] * len(lq), hq=hq, hkv=hkv, d=d, page=64, seed=21, t5=T5D, std=std)
    if low < 0:
        t.p.bias[28:] = low
        out, lse = t.run()
        assert _errors() == 0
        _check(t, out, lse, low)
        t.p.bias[:] = low
    else:  # the others are masked instead
        t.p.bias[28:] += low
    out, lse = t.run()
    got, gl = _wide(out[:t.p.total]), lse.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(gl / low - 1) < 1e-6).all()
    assert (np.abs(got) <= np.nanmax(np.abs(_wide(t.p.vc))) * (1 + 2.0 ** -7)).all()
