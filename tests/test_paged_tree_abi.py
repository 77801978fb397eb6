"""Trees of drafted tokens without a GPU: what is refused on the host through the C ABI, and the reference
against chains, for which it is the causal attention's."""
import ctypes

import numpy as np
import pytest

import attention_relative_position_gb300 as fa
from attention_relative_position_gb300 import _build
from exact_buckets import exact_bucket_array
from oracle import paged

FAKE = 1 << 20  # aligned non-null host value; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def test_exports(lib):
    for name in ("fat_paged_tree_plan", "fat_paged_tree_attn"):
        assert hasattr(lib, name) and hasattr(fa, name) and name in fa.__all__, name


def _plan(lib, ptrs=None, **kw):
    s = dict(total_q=10, num_seqs=2, max_seqlen_q=40, mask_words=2)
    s.update(kw)
    p = [FAKE + (i << 16) for i in range(5)]
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fat_paged_tree_plan(fa._TreeShape(*s.values(), None), *p)


def test_plan_refusals(lib):
    assert lib.fat_paged_tree_plan(None, *[FAKE] * 5) == -1
    for i in range(5):  # every array of this problem is needed, and 4-byte aligned
        assert _plan(lib, {i: None}) == -1, i
        assert _plan(lib, {i: FAKE + (i << 16) + 2}) == -2, i
    for bad in (dict(total_q=-1), dict(num_seqs=-1), dict(max_seqlen_q=-1), dict(mask_words=1),
                dict(mask_words=-1), dict(max_seqlen_q=65)):
        assert _plan(lib, **bad) == -2, bad
    assert _plan(lib, max_seqlen_q=4097, mask_words=200) == -5
    assert _plan(lib, {i: None for i in range(5)}, total_q=0) == 0
    # results over another array: parents, cu_seqlens_q, seqlens_k, positions, tree_mask
    for i, at in ((3, FAKE), (3, FAKE + 36), (4, FAKE + (1 << 16) - 76), (4, FAKE + (2 << 16) + 4),
                  (3, FAKE + (4 << 16) + 76)):
        assert _plan(lib, {i: at}) == -2, (i, at)


def _attn(lib, ptrs=None, words=1, **kw):
    s = dict(total_q=10, num_seqs=2, max_seqlen_q=20, max_seqlen_k=100, num_heads_q=4, table_width=7)
    s.update(kw)
    c = fa._Cache(FAKE, FAKE, 8, 16, 2, 64, 16 * 2 * 64, 2 * 64, 64)
    # q, block_table, cu_seqlens_q, seqlens_k, positions, tree_mask
    p = [FAKE] * 6
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fat_paged_tree_attn(fa._PagedShape(*s.values(), None), c, *p, words, None, 0, 0, 0, None,
                                   1.0, FAKE, ctypes.c_size_t(1 << 40), FAKE, None)


def test_attention_refusals(lib):
    for i in range(6):
        assert _attn(lib, {i: None}) == -1, i
        assert _attn(lib, {i: FAKE + (8 if i == 0 else 2)}) == -2, i
    assert _attn(lib, words=0) == -2
    assert _attn(lib, max_seqlen_q=33) == -2 and _attn(lib, max_seqlen_q=2 ** 31 - 1) == -2
    assert _attn(lib, total_q=0) == 0 and _attn(lib, num_seqs=0) == 0


@pytest.mark.parametrize("t5", [(32, 128, False), (64, 1024, True)])
def test_reference_of_chains(t5):
    rng = np.random.default_rng(2)
    lq, lk, hq, hkv, d, page = [5, 40, 1], [200, 40, 17], 4, 2, 64, 16
    pages = [-(-x // page) for x in lk]
    order = rng.permutation(sum(pages))
    table = np.zeros((3, max(pages)), np.int64)
    at = 0
    for i in range(3):
        table[i, :pages[i]] = order[at:at + pages[i]]
        at += pages[i]
    kc, vc = (rng.normal(size=(sum(pages), page, hkv, d)) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(lq)])
    q = rng.normal(size=(cu[-1], hq, d))
    bias, slopes = rng.normal(size=(t5[0], hq)), 2.0 ** -np.arange(1, hq + 1)
    parents = np.concatenate([np.arange(m) - 1 for m in lq])
    pos, mask = paged.tree_plan(parents, cu, lk, cu[-1], 40, 2)
    assert pos.tolist() == [k - m + j for m, k in zip(lq, lk) for j in range(m)]
    got = paged.tree_attention(q, kc, vc, table, cu, lk, pos, mask, bias=bias,
                               bucket=lambda x: exact_bucket_array(x, *t5), slopes=slopes, scale=0.1)
    # (the packed oracle takes table and slopes in fp32)
    want = paged.attention(q, kc, vc, table, cu, lk, table=bias.astype(np.float32), num_buckets=t5[0],
                           max_distance=t5[1], bidirectional=t5[2], slopes=slopes, causal=True,
                           scale=0.1)
    np.testing.assert_allclose(got[0], want[0], atol=2e-6)
    np.testing.assert_allclose(got[1], want[1], atol=2e-6)


def test_reference_of_a_tree():
    # one request: 2 cached keys; nodes 0 - 1, 0 - 2, 2 - 3; a fifth follows the context
    parents, cu, lk = [-1, 0, 0, 2, -1], [0, 5], [7]
    pos, mask = paged.tree_plan(parents, cu, lk, 6, 5, 1)
    assert pos.tolist() == [2, 3, 3, 4, 2, 0]
    assert mask[:, 0].tolist() == [1, 3, 5, 13, 16, 0]
    rng = np.random.default_rng(4)
    k, v = (rng.normal(size=(1, 16, 1, 8)) for _ in range(2))
    q = rng.normal(size=(5, 1, 8))
    out, lse, _, _, _ = paged.tree_attention(q, k, v, np.zeros((1, 1), int), cu, lk, pos, mask)
    for j, seen in enumerate([[0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 4], [0, 1, 2, 4, 5], [0, 1, 6]]):
        x = k[0, seen, 0] @ q[j, 0]
        assert np.isclose(lse[0, j], np.log(np.exp(x).sum()))
        assert np.allclose(out[j, 0], (np.exp(x) / np.exp(x).sum()) @ v[0, seen, 0])
