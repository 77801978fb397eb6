"""GPU parity of trees of drafted tokens over a paged cache: their maps (exact) and attention against the
fp64 oracle, then a step of verification that uses them together with append and the vocabulary's scores."""
import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa
from exact_buckets import exact_bucket_array
from oracle import linear_ce, paged
from test_gpu_paged import Problem, _bf16, _errors, _i32, _wide

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    _errors()


def _parents(rng, lq, reach, roots=0.0):
    out = []
    for m in lq:
        j = np.arange(m)
        p = j - 1 - np.minimum(rng.integers(0, reach, m), np.maximum(j - 1, 0))
        out.append(np.where((j == 0) | (rng.random(m) < roots), -1, p))
    return np.concatenate(out).astype(np.int64) if len(lq) else np.zeros(0, np.int64)


# ---- maps ---------------------------------------------------------------------------------------------
def _check_plan(parents, lq, lk, pad=0, most=None, bits=0, words=None):
    cu = np.concatenate([[0], np.cumsum(lq)])
    total = int(cu[-1]) + pad
    par = np.concatenate([parents, np.full(pad, 12345)])
    most = max(lq, default=0) if most is None else most
    w = -(-most // 32) if words is None else words
    want = paged.tree_plan(par, cu, lk, total, most, w)
    kw = {}
    if words is not None:
        kw["tree_mask"] = torch.full((total, w), -1, dtype=torch.int32, device=DEV)
    got = fa.fat_paged_tree_plan(_i32(par), _i32(cu), _i32(lk), most, **kw)
    assert _errors() == bits
    for name, g, x in zip(("positions", "mask"), got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), x, err_msg=name)
    return got


@pytest.mark.parametrize("lq,reach,pad,words", [
    ([1], 1, 0, None), ([5, 0, 1, 32, 33], 3, 3, None), ([64] * 16, 8, 0, None), ([31, 32, 33, 1], 1, 9, 4),
    ([500, 129, 128, 127], 2, 700, None), ([4096], 1, 1, None), ([4096, 7], 5, 0, 130),
    ([3] * 1500, 2, 5, None), ([0, 0], 1, 4, None)])
def test_plan(lq, reach, pad, words):
    rng = np.random.default_rng(len(lq) + reach)
    lk = np.array(lq) + rng.integers(0, 1000, len(lq))
    _check_plan(_parents(rng, lq, reach, 0.1), lq, lk, pad, words=words)


def test_plan_bad_input():
    rng = np.random.default_rng(3)
    lq = [9, 4, 20, 6]
    lk = np.array(lq) + 10
    par = _parents(rng, lq, 3)
    for bad in (9, 5, 100, -2, 2 ** 31 - 1, -(2 ** 31)):  # node 5's parent: itself, later ones, below -1
        p = par.copy()
        p[5] = bad
        _check_plan(p, lq, lk, bits=fa.FAT_DEVERR_INDEX)
    short = lk.copy()
    short[2] = 19
    _check_plan(par, lq, short, bits=fa.FAT_DEVERR_SEQLENS)
    _check_plan(par, lq, lk, most=19, bits=fa.FAT_DEVERR_SEQLENS)
    # corrupt row bounds: the other requests' rows are right, nothing is written outside the arrays
    cu = np.concatenate([[0], np.cumsum(lq)])
    for i, v in ((1, -3), (2, 1000), (2, 3), (4, 1000)):
        c = cu.copy()
        c[i] = v
        pos = torch.full((39,), -9, dtype=torch.int32, device=DEV)
        fa.fat_paged_tree_plan(_i32(par), _i32(c), _i32(lk), 20, positions=pos)
        assert _errors() & fa.FAT_DEVERR_SEQLENS


def test_plan_empty():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    pos, mask = fa.fat_paged_tree_plan(e, _i32([0]), e, 0)
    assert pos.shape == (0,) and mask.shape == (0, 0) and _errors() == 0
    # rows without a request
    pos, mask = fa.fat_paged_tree_plan(_i32([7, 7, 7]), _i32([0]), e, 40)
    assert pos.tolist() == [0] * 3 and (mask == 0).all() and mask.shape == (3, 2) and _errors() == 0


# ---- attention ----------------------------------------------------------------------------------------
class Tree:
    def __init__(self, lq, ctx, reach=3, roots=0.0, seed=0, mask=None, words=None, **kw):
        rng = np.random.default_rng(seed + 77)
        self.p = Problem(lq, np.array(lq) + np.array(ctx), causal=False, seed=seed, **kw)
        self.most = max(lq, default=0)
        self.words = -(-self.most // 32) if words is None else words
        self.pos, self.mask = paged.tree_plan(_parents(rng, lq, reach, roots), self.p.cu, self.p.lk,
                                              self.p.total, self.most, self.words)
        if mask == "random":  # any pattern, rows without a bit among them
            bits = rng.random((self.p.total, 32 * self.words)) < rng.choice([0, 0.1, 0.9],
                                                                            (self.p.total, 1))
            packed = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
            self.mask = packed.reshape(self.p.total, self.words).view(np.int32)

    def run(self, max_q=None, max_k=None, arrays=None, positions=None, mask=None, **kw):
        p = self.p
        extra = p.kwargs()
        del extra["causal"]
        max_q = self.most if max_q is None else max_q
        max_k = int(max(p.lk, default=0)) if max_k is None else max_k
        return fa.fat_paged_tree_attn(
            p.q, p.kc, p.vc, *(arrays or p.arrays()), _i32(self.pos) if positions is None else positions,
            _i32(self.mask) if mask is None else mask, max_q, max_k, **extra, **kw)

    def oracle(self, pos=None):
        p = self.p
        t5 = p.t5
        return paged.tree_attention(
            _wide(p.q), _wide(p.kc), _wide(p.vc), p.table, p.cu, p.lk, self.pos if pos is None else pos,
            self.mask, bias=None if p.bias is None else _wide(p.bias),
            bucket=(lambda d: exact_bucket_array(d, *t5)) if t5 else None,
            slopes=None if p.slopes is None else _wide(p.slopes), scale=p.scale)

    # Tolerances as of the attention of chains: a logit is formed in fp32 (d products, scale, bias), every
    # weight carries its error and the exponential's and is rounded to bf16, the output is rounded once.
    def check(self, out, lse, rows=None, pos=None):
        p = self.p
        ro, rl, a, s, b = self.oracle(pos)
        ex = (p.d * s + 4 * (s + b)) * 2.0 ** -24
        got, gl = _wide(out[:p.total]), lse.cpu().numpy()[:, :p.total].astype(np.float64)
        if rows is not None:
            got, ro, a, gl, rl = got[rows], ro[rows], a[rows], gl[:, rows], rl[:, rows]
        tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ex + 2.0 ** -18) * a * 1.01 + 1e-30
        err = np.abs(got - ro)
        assert (err <= tol).all(), (err / tol).max()
        fin = np.isfinite(rl)
        assert np.array_equal(np.isfinite(gl), fin) and (gl[~fin] == -np.inf).all()
        assert (got.transpose(1, 0, 2)[~fin] == 0).all()
        ltol = ex + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl[fin])
        assert (np.abs(gl[fin] - rl[fin]) <= ltol).all(), np.abs(gl[fin] - rl[fin]).max()


T5D, T5B = (32, 128, False), (64, 1024, True)
CASES = {
    "one_node": dict(lq=[1], ctx=[0], hq=1, hkv=1, d=64, page=16),
    "no_context": dict(lq=[7, 16, 1], ctx=[0, 0, 0], hq=2, hkv=2, d=64, page=16, t5=T5D),
    "few_page_edges": dict(lq=[5] * 8, ctx=[10, 11, 12, 27, 28, 59, 60, 123], hq=2, hkv=2, d=64, page=16,
                           t5=T5D, alibi=True),
    "few_d128_group4": dict(lq=[4, 3, 1, 2, 0, 4], ctx=[1200, 0, 9, 130, 7, 4000], hq=8, hkv=2, d=128,
                            page=16, t5=T5D, reach=2),
    "few_bidir": dict(lq=[16, 13], ctx=[900, 1500], hq=3, hkv=3, d=64, page=64, t5=T5B, reach=1),
    "few_random": dict(lq=[16, 9, 2], ctx=[0, 300, 0], hq=4, hkv=4, d=128, page=32, mask="random",
                       alibi=True, words=2),
    "tile_group1": dict(lq=[60, 17, 128], ctx=[700, 0, 1], hq=2, hkv=2, d=64, page=32, t5=T5D),
    "tile_chain": dict(lq=[130, 40], ctx=[100, 2000], hq=2, hkv=1, d=128, page=16, reach=1, t5=T5D,
                       alibi=True),
    "tile_large": dict(lq=[300, 129], ctx=[900, 37], hq=3, hkv=3, d=64, page=128, t5=T5B, reach=4,
                       roots=0.02),
    "tile_large_d128": dict(lq=[270], ctx=[1111], hq=2, hkv=2, d=128, page=64, alibi=True, reach=6),
    "tile_group4": dict(lq=[61, 24, 33], ctx=[3000, 128, 127], hq=8, hkv=2, d=128, page=64, reach=8),
    "tile_group5": dict(lq=[26, 11], ctx=[500, 90], hq=10, hkv=2, d=128, page=16, alibi=True, roots=0.3),
    "tile_group100": dict(lq=[5, 2], ctx=[300, 0], hq=100, hkv=1, d=64, page=32, t5=T5D),
    "tile_random": dict(lq=[70, 33], ctx=[0, 65], hq=4, hkv=2, d=128, page=16, mask="random", t5=T5D,
                        words=5),
    "tile_random_d64": dict(lq=[200, 64], ctx=[0, 0], hq=2, hkv=2, d=64, page=16, mask="random",
                            t5=T5B, alibi=True),
    # requests of as many rows each, more blocks of 128 rows than SMs
    "many": dict(lq=[140] * 12, ctx=[0, 1, 127, 128, 129, 300, 500, 700, 5, 60, 70, 900], hq=8, hkv=8,
                 d=64, page=16, t5=T5D, reach=4),
    "many_d128": dict(lq=[80] * 13, ctx=[0, 1100, 48, 47, 49, 300, 500, 700, 5, 60, 70, 9, 600], hq=16,
                      hkv=8, d=128, page=64, alibi=True, reach=3),
    "many_random": dict(lq=[150] * 40, ctx=[0] * 39 + [1200], hq=2, hkv=2, d=64, page=64, mask="random",
                        t5=T5B),
    # three tiles of own keys: rows that see nothing in the first tiles taken
    "random_long": dict(lq=[300, 380, 2], ctx=[0, 0, 200], hq=2, hkv=2, d=128, page=16, mask="random"),
    "mixed": dict(lq=[1, 60, 3, 0, 16, 40], ctx=[2000, 30, 1000, 5, 800, 4000], hq=8, hkv=2, d=64,
                  page=16, t5=T5D),
    "mixed_d128": dict(lq=[1, 50, 4, 1], ctx=[700, 1300, 0, 5000], hq=16, hkv=4, d=128, page=128,
                       alibi=True),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    t = Tree(seed=len(name), **CASES[name])
    out, lse = t.run()
    assert _errors() == 0
    t.check(out, lse)


# Logits of hundreds: the first reference of a row is passed by far more than 2^32 in later tiles, again and
# again, and whole tiles vanish beside others.
@pytest.mark.parametrize("std", [3.0, 12.0])
@pytest.mark.parametrize("lq,hq,hkv,d", [([60, 17], 2, 2, 64), ([128], 2, 2, 128), ([30, 32], 8, 4, 128),
                                         ([5], 6, 2, 128), ([140] * 12, 8, 8, 64)])
def test_large_logits(std, lq, hq, hkv, d):
    t = Tree(lq, [1500, 800] + [100] * 10 if len(lq) > 2 else [1500, 800][:len(lq)], hq=hq, hkv=hkv, d=d,
             page=64, std=std, seed=3, alibi=True)
    t.check(*t.run())


@pytest.mark.parametrize("low", [-float("inf"), float(np.finfo(np.float32).min), -1e38])
@pytest.mark.parametrize("lq,ctx,hq,hkv,d", [([5, 3], [40, 3], 2, 2, 64), ([40, 20], [700, 9], 2, 1, 64),
                                             ([61], [300], 4, 2, 128), ([140] * 12, [90] * 12, 8, 8, 64)])
def test_bias_that_masks(low, lq, ctx, hq, hkv, d):
    """T5 buckets whose bias is -infinity, the lowest fp32 value, or far below every logit: keys there get no
    weight beside any other key; a row of such keys alone gets none (or, at -1e38, the softmax of its biases:
    all equal to fp32, so that every key it sees gets the same weight)."""
    t = Tree(lq, ctx, hq=hq, hkv=hkv, d=d, page=16, t5=T5D, seed=2)
    p = t.p
    p.bias[:, 0] = low            # head 0: every key
    p.bias[1:9, 1] = low          # head 1: distances 1 to 8
    out, lse = t.run()
    assert _errors() == 0
    p.bias[p.bias < -2e38] = -float("inf")
    ro, rl, a, s, b = t.oracle()
    got, gl = _wide(out), lse.double().cpu().numpy()
    if low < -2e38:
        assert (gl[0] == -np.inf).all() and (got[:, 0] == 0).all()
    else:
        assert (np.abs(gl[0] / low - 1) < 1e-6).all()
    heads = np.arange(1, p.hq)
    fin = np.isfinite(p.bias.cpu().numpy()) & (p.bias.cpu().numpy() > -1e37)
    big = float(np.abs(p.bias.cpu().numpy()[fin]).max())
    ex = (p.d * s + 4 * (s + big)) * 2.0 ** -24
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ex + 2.0 ** -18) * a * 1.01 + 1e-30
    assert (np.abs(got - ro)[:, heads] <= tol[:, heads]).all()
    ok = rl[heads] > -1e37
    assert (np.abs(gl[heads] - rl[heads])[ok] <= (ex + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl[heads]))[ok]).all()


@pytest.mark.parametrize("layout", ["head", "block"])
@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group4"])
def test_cache_layouts(layout, name):
    t = Tree(seed=5, layout=layout, **CASES[name])
    t.check(*t.run())


@pytest.mark.parametrize("lq,hq,hkv,d", [([5, 3], 6, 2, 64), ([7], 2, 2, 128), ([60, 20], 8, 2, 128),
                                         ([150, 1], 4, 2, 64)])
def test_a_chain_is_causal_attention(lq, hq, hkv, d):
    t = Tree(lq, [700, 33][:len(lq)], reach=1, hq=hq, hkv=hkv, d=d, page=16, t5=T5D, alibi=True, seed=8)
    out, lse = t.run()
    t.p.causal = True
    t.p.check(out, lse)  # against the oracle of the packed attention


@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group4", "mixed"])
def test_rows_behind_and_larger_bounds(name):
    t = Tree(seed=6, pad=9, words=7, **CASES[name])
    p = t.p
    pad = np.full((9,), 1 << 30), np.full((9, 7), -1)
    out, lse = torch.full_like(p.q, 3.0), torch.full((p.hq, p.total + 9), 5.0, device=DEV)
    t.run(out=out, lse=lse, positions=_i32(np.concatenate([t.pos, pad[0]])),
          mask=_i32(np.concatenate([t.mask, pad[1]])), max_q=200, max_k=9000)
    assert _errors() == 0
    t.check(out, lse)
    assert (out[p.total:] == 3.0).all() and (lse[:, p.total:] == 5.0).all()


@pytest.mark.parametrize("name", ["few_bidir", "tile_group1", "tile_large", "tile_chain"])
def test_positions_outside_are_taken_as_the_nearest(name):
    t = Tree(seed=7, **CASES[name])
    pos = t.pos.copy()
    pos[2], pos[9] = -5, 2 ** 31 - 1
    pos[-1] = -(2 ** 31)
    out, lse = t.run(positions=_i32(pos))
    assert _errors() == fa.FAT_DEVERR_INDEX
    t.check(out, lse, pos=pos)


def test_corrupt_requests_are_left_out():
    t = Tree([3, 40, 2, 30], [50, 60, 500, 9], hq=4, hkv=2, d=64, page=16, seed=4, t5=T5D)
    p = t.p
    lk = p.lk.copy()
    lk[1], lk[2] = 39, 1  # fewer keys than queries
    out, lse = torch.full_like(p.q, 3.0), torch.full((4, p.total), 5.0, device=DEV)
    t.run(arrays=(_i32(p.table), _i32(p.cu), _i32(lk)), out=out, lse=lse)
    assert _errors() == fa.FAT_DEVERR_SEQLENS
    rows = np.r_[0:3, 45:75]
    t.check(out, lse, rows=rows)
    assert (out[3:45] == 3.0).all() and (lse[:, 3:45] == 5.0).all()


@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group4", "tile_large", "mixed_d128"])
def test_captured_and_replayed(name):
    """One capture, replayed with another tree of the same lengths; repeated calls agree bit for bit."""
    a, b = (Tree(seed=9, **dict(CASES[name], reach=r)) for r in (2, 5))
    pos, mask = _i32(a.pos), _i32(a.mask)
    arrays = a.p.arrays()
    ws = torch.empty(max(1, fa.fat_paged_attn_workspace_size(a.p.q, a.p.kc, arrays[1], a.most, 6000)),
                     dtype=torch.uint8, device=DEV)
    out, lse = torch.zeros_like(a.p.q), torch.zeros((a.p.hq, a.p.total), device=DEV)

    def call():
        a.run(arrays=arrays, positions=pos, mask=mask, max_k=6000, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in (b, a, b):
        pos.copy_(_i32(x.pos))
        mask.copy_(_i32(x.mask))
        g.replay()
        assert _errors() == 0
        a.pos, a.mask = x.pos, x.mask
        a.check(out, lse)
        want = out.clone()
        call()
        assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group1", "tile_group4", "many"])
def test_watchdog(name):
    """No copies are issued: the waits run out, the status says so, and the next call is right."""
    t = Tree(seed=33, **CASES[name])
    try:
        fa.fat_attn_debug_set_watchdog(50_000_000, 1)
        t.run()
        assert _errors() == fa.FAT_DEVERR_TIMEOUT_FWD
    finally:
        fa.fat_attn_debug_set_watchdog(0, 0)
    t.check(*t.run())
    assert _errors() == 0


@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group4", "tile_large", "many", "mixed_d128"])
def test_workspace_of_the_given_size(name):
    """Nothing is written behind the bytes that the size names, whatever they held."""
    t = Tree(seed=12, **CASES[name])
    p = t.p
    size = fa.fat_paged_attn_workspace_size(p.q, p.kc, _i32(p.cu), t.most, 2000)
    buf = torch.full((size + 4096,), 0xff, dtype=torch.uint8, device=DEV)
    k = int(max(p.lk))
    t.check(*t.run(max_k=max(2000, k), workspace=buf[:size] if k <= 2000 else None))
    assert (buf[size:] == 0xff).all() and _errors() == 0


@pytest.mark.parametrize("name", ["few_d128_group4", "tile_group4", "tile_group1", "many"])
@pytest.mark.parametrize("bad", [-1, 1 << 20])
def test_bad_page_counts_as_zeros(name, bad):
    t = Tree(seed=14, **CASES[name])
    p = t.p
    i = int(np.argmax(p.lk))
    p.table[i, 0] = bad
    out, lse = t.run()
    assert _errors() == fa.FAT_DEVERR_PAGES
    t.check(out, lse)


@pytest.mark.parametrize("name", ["few_page_edges", "tile_group1", "tile_group4", "many"])
def test_nan_shows_in_its_rows(name):
    t = Tree(seed=15, **CASES[name])
    p = t.p
    clean, clean_lse = t.run()
    p.q[2, 0] = float("nan")
    out, lse = t.run()
    assert torch.isnan(out[2, 0]).all() and torch.isnan(lse[0, 2])
    keep = torch.ones_like(lse, dtype=torch.bool)
    keep[0, 2] = False
    # (the others: as before, but for what rows that share a vote do together)
    t.p.q[2, 0] = 0
    ro, rl, a, s, b = t.oracle()
    assert torch.isfinite(out.transpose(0, 1)[keep]).all()
    ex = (p.d * s + 4 * (s + b)) * 2.0 ** -24
    off = (lse[:, :p.total].double().cpu() - torch.from_numpy(rl)).abs()[keep[:, :p.total].cpu()]
    assert (off <= ex + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl).max()).all()


def test_two_calls_at_once():
    a, b = Tree(seed=16, **CASES["tile_group4"]), Tree(seed=17, **CASES["mixed"])
    want = [x.run() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [dict(arrays=x.p.arrays(), positions=_i32(x.pos), mask=_i32(x.mask)) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [x.run(stream=s, **k) for x, s, k in zip((a, b), streams, args)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_requests_share_pages():
    """The same context pages under two trees."""
    t = Tree([20, 20], [256, 256], hq=4, hkv=2, d=64, page=64, seed=18)
    p = t.p
    p.table[1, :4] = p.table[0, :4]
    t.check(*t.run())


def test_arguments_are_checked():
    t = Tree(seed=1, **CASES["tile_group4"])
    pos, mask = _i32(t.pos), _i32(t.mask)
    for kw, err in ((dict(positions=pos[:-1]), ValueError), (dict(positions=pos.long()), TypeError),
                    (dict(mask=mask[:-1]), ValueError), (dict(mask=mask.float()), TypeError),
                    (dict(mask=mask.cpu()), ValueError), (dict(mask=mask[:, :1]), (fa.FatAttnError, ValueError)),
                    (dict(max_q=65), fa.FatAttnError), (dict(mask=mask.t()), ValueError),
                    (dict(positions=None, mask=mask.flatten()), ValueError)):
        with pytest.raises(err):
            t.run(**kw)
    par = _i32(np.zeros(5))
    for args, err in (((par.long(), _i32([0, 5]), _i32([9]), 5), TypeError),
                      ((par, _i32([0]), _i32([9]), 5), ValueError),
                      ((par, _i32([0, 5]), _i32([9]), -1), fa.FatAttnError),
                      ((par, _i32([0, 5]), _i32([9]), 4097), fa.FatAttnError),
                      ((par, _i32([0, 5]), _i32([9]), 5, _i32(np.zeros(4))), ValueError),
                      ((par, _i32([0, 5]), _i32([9]), 33, None, _i32(np.zeros((5, 1)))), fa.FatAttnError),
                      ((par, _i32([0, 5]), _i32([9]), 5, par), fa.FatAttnError)):
        with pytest.raises(err):
            fa.fat_paged_tree_plan(*args)
    assert _errors() == 0


# ---- a step of verification ---------------------------------------------------------------------------
@pytest.mark.parametrize("graph", [False, True])
def test_verification_step(graph):
    """Plan, the trees' maps, append at their positions, attention over them, and the scores of the drafted
    tokens: every path gets what a plain chain of its tokens would get."""
    rng = np.random.default_rng(12)
    hq, hkv, d, page, vocab = 4, 2, 64, 16, 3001
    ctx, lq = [75, 0, 130], [13, 9, 40]
    n, total, cap = 3, 62, 70
    pages = 64
    par = _parents(rng, lq, 4)
    kc, vc = (torch.full((pages, page, hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    free = _i32(rng.permutation(pages))
    table = torch.full((n, 12), -1, dtype=torch.int32, device=DEV)
    rope = fa.fat_rope_init(d)
    docs = _bf16(rng, sum(ctx), hq + 2 * hkv, d)
    new = torch.full((cap, hq + 2 * hkv, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    new[:total] = _bf16(rng, total, hq + 2 * hkv, d)
    weight = _bf16(rng, vocab, hq * d, std=0.2)
    drafted = _i32(rng.integers(0, vocab, cap))
    parents = _i32(np.concatenate([par, np.full(8, -1)]))
    # the contexts first
    cu0, lk0, pos0, slots0, counts = fa.fat_paged_plan(_i32([0] * n), _i32(ctx), free, table, page, pages,
                                                       sum(ctx))
    q, k, v = docs.split([hq, hkv, hkv], dim=1)
    fa.fat_paged_append(k, v, kc, vc, slots0, positions=pos0, rope=rope)
    free = free[int(counts[0]):].contiguous()
    res = {}

    def step():
        cu, lk, _, slots, _ = fa.fat_paged_plan(_i32_ctx, _i32_new, free, table, page, pages, cap)
        pos, mask = fa.fat_paged_tree_plan(parents, cu, lk, 64)
        q, k, v = new.split([hq, hkv, hkv], dim=1)
        qr = fa.fat_paged_append(k, v, kc, vc, slots, q=q, positions=pos, rope=rope)
        out, _ = fa.fat_paged_tree_attn(qr, kc, vc, table, cu, lk, pos, mask, 64, 256,
                                        softmax_scale=d ** -0.5)
        loss, _ = fa.fat_linear_cross_entropy_fwd(out.view(cap, hq * d), weight, drafted)
        res.update(out=out, loss=loss, pos=pos, mask=mask)

    _i32_ctx, _i32_new = _i32(ctx), _i32(lq)
    saved = table.clone()
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        table.copy_(saved)
        g.replay()
    else:
        step()
    assert _errors() == 0
    out, loss = res["out"][:total], res["loss"][:total]
    # every node: its request's context and its path as one chain, through the packed attention
    at_ctx = np.concatenate([[0], np.cumsum(ctx)])
    cu = np.concatenate([[0], np.cumsum(lq)])
    rows, lens, pos, ends = [], [], [], []
    for i in range(n):
        for j in range(lq[i]):
            path, a = [], j
            while a >= 0:
                path.insert(0, a)
                a = int(par[cu[i] + a])
            rows.append(torch.cat([docs[at_ctx[i]:at_ctx[i + 1]], new[[int(cu[i]) + b for b in path]]]))
            lens.append(len(rows[-1]))
            ends.append(sum(lens) - 1)
            assert int(res["pos"][cu[i] + j]) == lens[-1] - 1
    packed = torch.cat(rows)
    cus = _i32(np.concatenate([[0], np.cumsum(lens)]))
    qr, kr = (fa.fat_rope_apply(x.contiguous(), cus, max(lens))
              for x in (packed[:, :hq], packed[:, hq:hq + hkv]))
    # RoPE of the append turns pairs (2i, 2i + 1) by default as the packed call does
    want, _ = fa.fat_xattn_fwd(qr, kr, packed[:, hq + hkv:].contiguous(), cus, cus, max(lens), max(lens),
                               causal=True, softmax_scale=d ** -0.5)
    want = want[ends]
    # both are within a bf16 rounding of P and of the result of the same exact values
    most = packed[:, hq + hkv:].double().abs().amax()
    assert ((out.double() - want.double()).abs() <= 2.0 ** -8 * 2 * (want.double().abs() + most)).all()
    score, _ = linear_ce.forward(out.reshape(total, hq * d), weight, drafted[:total])
    # a logit: 256 products of bf16 values in fp32
    tol = 2.1 * (256 / 16 + 16) * 2.0 ** -23 * float((out.reshape(total, -1).double().abs()
                                                     @ weight.double().abs().t()).max()) + 1e-4
    assert (loss.double() - score).abs().max() <= tol


# Items over most of the grid (more parts than a warp's task holds), a few parts beside whole items, and parts of
# requests that begin where another ends; 64 and 128 rows, a group of rows that a warpgroup has none of.
@pytest.mark.parametrize("lq,ctx,hq,hkv,d", [
    ([30], [11000], 2, 2, 64), ([30], [9000], 4, 2, 128), ([100], [9001], 1, 1, 64), ([70], [8900], 1, 1, 128),
    ([25, 3, 30], [4000, 20, 5003], 2, 1, 128), ([17, 40, 64, 20], [2000, 1999, 30, 2500], 4, 2, 64),
    ([20] * 9, [1100 + 130 * i for i in range(9)], 6, 2, 128)])
def test_long_contexts_in_parts(lq, ctx, hq, hkv, d):
    t = Tree(lq, ctx, hq=hq, hkv=hkv, d=d, page=64, seed=21, alibi=True)
    size = fa.fat_paged_attn_workspace_size(t.p.q, t.p.kc, _i32(t.p.cu), t.most, int(max(t.p.lk)))
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    out, lse = t.run(workspace=ws)
    assert _errors() == 0
    t.check(out, lse)
    again, lse2 = t.run(workspace=ws)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# More requests than a block has threads, and more in a CTA's stretch than it stages; few rows and many.
@pytest.mark.parametrize("lq,hq,d", [([20, 1, 3] + [1, 2] * 700 + [0, 17], 2, 128), ([1] * 10500 + [33], 1, 64),
                                     ([1, 2] * 3000 + [4], 2, 64)])
def test_many_requests(lq, hq, d):
    t = Tree(lq, [(5 * i) % 23 for i in range(len(lq))], hq=hq, hkv=1, d=d, page=16, seed=13)
    out, lse = t.run()
    assert _errors() == 0
    t.check(out, lse)
