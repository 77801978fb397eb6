"""Argument checks of the paged-cache calls: what is refused on the host, before anything is
enqueued, through the C ABI (no GPU needed)."""
import ctypes

import pytest

import attention_relative_position_gb300 as fa
from attention_relative_position_gb300 import _build

FAKE = 1 << 20  # aligned non-null host value; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def test_exports(lib):
    for name in ("fat_paged_plan", "fat_rope_init", "fat_rope_embed", "fat_paged_append",
                 "fat_paged_attn", "fat_paged_attn_workspace_size"):
        assert hasattr(lib, name) and hasattr(fa, name), name


def _plan(lib, ptrs=None, **kw):
    s = dict(num_seqs=2, page_size=16, num_pages=8, table_width=4, num_free=3, max_tokens=5)
    s.update(kw)
    p = [FAKE] * 9
    for i, v in (ptrs or {}).items():
        p[i] = v
    return lib.fat_paged_plan(fa._PlanShape(*s.values(), None), *p)


def test_plan_refusals(lib):
    assert lib.fat_paged_plan(None, *[FAKE] * 9) == -1
    for i in range(9):  # every array of this problem is needed, and 4-byte aligned
        assert _plan(lib, {i: None}) == -1, i
        assert _plan(lib, {i: FAKE + 2}) == -2, i
    for bad in (dict(num_seqs=-1), dict(page_size=0), dict(page_size=8), dict(page_size=48),
                dict(page_size=1 << 17), dict(num_pages=0), dict(table_width=-1),
                dict(num_free=-1), dict(max_tokens=-1), dict(num_pages=1 << 27, page_size=16)):
        assert _plan(lib, **bad) == -2, bad


def test_rope_init_refusals_and_rates():
    for kw in (dict(rotary_dim=0), dict(rotary_dim=8), dict(rotary_dim=24), dict(rotary_dim=272),
               dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, base=float("inf")),
               dict(rotary_dim=64, base=float("nan")), dict(rotary_dim=64, factor=0.0),
               dict(rotary_dim=64, factor=-2.0), dict(rotary_dim=64, amplitude=0.0),
               dict(rotary_dim=64, amplitude=1e300), dict(rotary_dim=64, ramp=(4.0, 1.0, 4096.0)),
               dict(rotary_dim=64, ramp=(1.0, 1.0, 4096.0)),
               dict(rotary_dim=64, ramp=(-1.0, 4.0, 4096.0)),
               dict(rotary_dim=64, ramp=(1.0, 4.0, -1.0))):
        with pytest.raises(fa.FatAttnError) as e:
            fa.fat_rope_init(**kw)
        assert e.value.code == -2, kw
    import math
    from oracle import paged
    for kw in (dict(), dict(factor=4.0), dict(base=500000.0, factor=8.0, ramp=(1.0, 4.0, 8192.0)),
               dict(factor=0.25)):
        r = fa.fat_rope_init(96, **kw)
        want = paged.rope_angles([1.0], 96, **kw)[0] / (2 * math.pi)
        for i in range(48):
            # doubles on both sides: a few roundings of 2^-53 relative, 2^-53 of the fraction
            assert abs(r.rate[i] / 2.0 ** 64 - (want[i] - math.floor(want[i]))) \
                <= 16 * 2.0 ** -53 * max(1.0, want[i])


def _embed(lib, rope, x=FAKE, y=FAKE + 4096, pos=FAKE, tokens=4, heads=2, d=64, xs=(128, 64),
           ys=(128, 64)):
    sh = fa._RopeShape(tokens, heads, d, *xs, *ys, None)
    return lib.fat_rope_embed(sh, rope, x, y, pos, 0)


def test_rope_embed_refusals(lib):
    r = fa.fat_rope_init(64)
    assert lib.fat_rope_embed(None, r, FAKE, FAKE, FAKE, 0) == -1
    assert _embed(lib, None) == -1
    assert _embed(lib, r, x=None) == -1 and _embed(lib, r, y=None) == -1
    assert _embed(lib, r, pos=None) == -1
    assert _embed(lib, r, x=FAKE + 8) == -2 and _embed(lib, r, y=FAKE + 2) == -2
    assert _embed(lib, r, pos=FAKE + 2) == -2
    assert _embed(lib, r, tokens=-1) == -2 and _embed(lib, r, heads=0) == -2
    assert _embed(lib, r, d=60) == -2
    assert _embed(lib, r, d=32) == -2  # fewer channels than the rotation
    assert _embed(lib, r, xs=(132, 64)) == -2 and _embed(lib, r, xs=(-128, 64)) == -2
    assert _embed(lib, r, ys=(128, 32)) == -2  # rows of y that overlap
    assert _embed(lib, r, ys=(0, 64)) == -2
    assert _embed(lib, r, x=FAKE, y=FAKE, xs=(256, 64)) == -2  # in place with other strides
    assert _embed(lib, fa._Rope()) == -2  # a record that fat_rope_init has not filled
    assert _embed(lib, r, tokens=0) == 0


def _cache(**kw):
    c = dict(k=FAKE, v=FAKE, num_pages=8, page_size=16, num_heads=2, head_dim=64,
             stride_page=2048, stride_token=128, stride_head=64)
    c.update(kw)
    return fa._Cache(*c.values())


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(num_pages=0), -2),
              (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(page_size=1 << 17), -2),
              (dict(num_heads=0), -2), (dict(head_dim=0), -2), (dict(head_dim=60), -2),
              (dict(k=FAKE + 8), -2), (dict(stride_page=2049), -2), (dict(stride_token=-128), -2),
              (dict(stride_head=32), -2), (dict(stride_token=0), -2), (dict(stride_page=0), -2),
              (dict(num_pages=1 << 28), -2)]


def _append(lib, cache, rope=None, q=None, k=FAKE, v=FAKE, pos=None, slots=FAKE, qo=None, tokens=3,
            hq=4, qs=(256, 64), ks=(128, 64), vs=(128, 64)):
    sh = fa._AppendShape(tokens, hq, *qs, *ks, *vs, None)
    return lib.fat_paged_append(sh, cache, rope, q, k, v, pos, slots, qo)


def test_append_refusals(lib):
    r = fa.fat_rope_init(64)
    for kw, code in BAD_CACHES:
        assert _append(lib, _cache(**kw)) == code, kw
    c = _cache()
    assert lib.fat_paged_append(None, c, None, None, FAKE, FAKE, None, FAKE, None) == -1
    assert _append(lib, None) == -1
    assert _append(lib, c, k=None) == -1 and _append(lib, c, v=None) == -1
    assert _append(lib, c, slots=None) == -1
    assert _append(lib, c, rope=r) == -1  # a rotation without positions
    assert _append(lib, c, q=FAKE) == -1 and _append(lib, c, qo=FAKE) == -1
    assert _append(lib, c, tokens=-1) == -2
    assert _append(lib, c, q=FAKE, qo=FAKE, hq=0) == -2
    assert _append(lib, c, q=FAKE, qo=FAKE, qs=(512, 64)) == -2  # in place, not contiguous
    assert _append(lib, c, q=FAKE, qo=FAKE + 4096, qs=(257, 64)) == -2
    assert _append(lib, c, ks=(129, 64)) == -2 and _append(lib, c, vs=(128, 63)) == -2
    assert _append(lib, c, k=FAKE + 8) == -2 and _append(lib, c, slots=FAKE + 2) == -2
    assert _append(lib, c, rope=fa.fat_rope_init(128), pos=FAKE) == -2
    assert _append(lib, c, rope=r, pos=FAKE + 1) == -2
    assert _append(lib, c, tokens=0) == 0


def _attn(lib, cache, ptrs=None, bias=None, nb=0, md=0, bidir=1, slopes=None, ws=FAKE,
          ws_bytes=1 << 40, **kw):
    s = dict(total_q=6, num_seqs=2, max_seqlen_q=3, max_seqlen_k=64, num_heads_q=4, table_width=4)
    s.update(kw)
    p = dict(q=FAKE, table=FAKE, cu=FAKE, lk=FAKE, out=FAKE, lse=FAKE)
    p.update(ptrs or {})
    return lib.fat_paged_attn(fa._PagedShape(*s.values(), None), cache, p["q"], p["table"],
                              p["cu"], p["lk"], bias, nb, md, bidir, slopes, 1, 0.125, ws,
                              ws_bytes, p["out"], p["lse"])


def test_attn_refusals(lib):
    for kw, code in BAD_CACHES:
        assert _attn(lib, _cache(**kw)) == code, kw
    c = _cache()
    assert _attn(lib, None) == -1
    for name in ("q", "table", "cu", "lk", "out"):
        assert _attn(lib, c, {name: None}) == -1, name
    for name, off in (("q", 8), ("table", 2), ("cu", 2), ("lk", 1), ("out", 8), ("lse", 4)):
        assert _attn(lib, c, {name: FAKE + off}) == -2, name
    for bad in (dict(total_q=-1), dict(num_seqs=-1), dict(max_seqlen_q=-1), dict(max_seqlen_k=-1),
                dict(num_heads_q=0), dict(num_heads_q=5), dict(table_width=-1)):
        assert _attn(lib, c, **bad) == -2, bad
    assert _attn(lib, _cache(head_dim=96, stride_head=96, stride_token=192, stride_page=4096)) == -2
    assert _attn(lib, c, num_heads_q=258) == -5  # 129 query heads per key/value head
    assert _attn(lib, c, num_seqs=70000) == -5
    assert _attn(lib, c, max_seqlen_k=(1 << 30) + 1) == -5
    # strides of which one is no multiple of the one before
    assert _attn(lib, _cache(stride_head=72, stride_token=200, stride_page=4000)) == -5
    assert _attn(lib, c, bias=FAKE, nb=31, md=128, bidir=1) == -3
    assert _attn(lib, c, bias=FAKE, nb=32, md=8, bidir=1) == -3
    assert _attn(lib, c, bias=FAKE, nb=32, md=40000, bidir=1) == -5  # saturates too far out
    assert _attn(lib, _cache(num_heads=1), bias=FAKE, nb=128, md=512, num_heads_q=64) == -5
    assert _attn(lib, c, bias=FAKE + 4, nb=32, md=128) == -2
    assert _attn(lib, c, slopes=FAKE + 4) == -2
    assert _attn(lib, c, ws=FAKE + 16) == -2
    # nothing to do: returns before touching the device
    for empty in (dict(total_q=0), dict(num_seqs=0), dict(max_seqlen_q=0)):
        assert _attn(lib, c, **empty) == 0, empty
    assert lib.fat_paged_attn_workspace_size(None, ctypes.byref(c)) == 0


def test_binding_refusals():
    """What the binding refuses before it reaches the library (which needs no GPU to say so)."""
    import torch
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    rope = fa.fat_rope_init(64)
    for err, call in (
            (TypeError, lambda: fa.fat_paged_plan([1], i, i, i.view(2, 1), 16, 2, 2)),
            (TypeError, lambda: fa.fat_paged_plan(i.long(), i, i, i.view(2, 1), 16, 2, 2)),
            (ValueError, lambda: fa.fat_paged_plan(i, i, i, i.view(2, 1), 16, 2, 2)),  # on the CPU
            (TypeError, lambda: fa.fat_rope_embed(x.float(), i, rope)),
            (ValueError, lambda: fa.fat_rope_embed(x, i, rope)),
            (TypeError, lambda: fa.fat_rope_embed(None, i, rope)),
            (ValueError, lambda: fa.fat_paged_append(x, x, cache, cache, i)),
            (TypeError, lambda: fa.fat_paged_append(x.half(), x, cache, cache, i)),
            (ValueError, lambda: fa.fat_paged_attn(x, cache, cache, i.view(2, 1), i, i, 1, 1)),
            (TypeError, lambda: fa.fat_paged_attn(1, cache, cache, i.view(2, 1), i, i, 1, 1)),
            (TypeError, lambda: fa.fat_paged_attn_workspace_size("q", cache, i, 1, 1))):
        with pytest.raises(err):
            call()
    with pytest.raises(TypeError):
        fa._load_calls().plan(1, 2)


OVERLAPPING = [dict(stride_token=64, stride_head=64),     # a token's second head, the next one's first
               dict(stride_head=256, stride_token=128),   # heads inside each other's tokens
               dict(stride_page=1024), dict(stride_page=64, stride_head=512)]
APART = [dict(), dict(num_heads=1, stride_head=0, stride_token=64, stride_page=1024),
         dict(stride_head=1024, stride_token=64),         # heads outside the tokens of a page
         dict(stride_page=64 * 6, stride_head=128, stride_token=64 * 6 * 8),  # pages inside tokens
         # one page of a block of several layers: its own stride says nothing
         dict(num_pages=1, stride_page=0, stride_head=4096, stride_token=64)]


@pytest.mark.parametrize("kw", OVERLAPPING)
def test_caches_whose_rows_overlap_are_refused(lib, kw):
    assert _append(lib, _cache(**kw)) == -2
    assert _attn(lib, _cache(**kw)) == -2


@pytest.mark.parametrize("kw", APART)
def test_caches_whose_rows_lie_apart_pass(lib, kw):
    assert _append(lib, _cache(**kw), tokens=0) == 0
    if "stride_page" not in kw or kw["stride_page"] in (0, 1024):
        assert _attn(lib, _cache(**kw), total_q=0) == 0
    else:  # attention wants the pages outermost
        assert _attn(lib, _cache(**kw), total_q=0) == -5


def test_rope_rows_of_the_result_lie_apart(lib):
    r = fa.fat_rope_init(64)
    assert _embed(lib, r, ys=(64, 64)) == -2
    assert _embed(lib, r, ys=(128, 128)) == -2
    assert _embed(lib, r, ys=(64, 192)) == -2
    assert _embed(lib, r, tokens=0, ys=(64, 256)) == 0


def test_register_splits_are_checked_before_a_launch():
    """A kernel whose warps raise their register share waits for registers that a build with fewer of
    them never frees: its launcher has to hand the split's need to prepare_kernel, which refuses such
    a build."""
    import glob
    import os
    import re
    found = {}
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu")):
        text = open(path).read()
        if not re.search(r"\bregs_inc<", text):
            continue
        calls = re.findall(r"\bprepare_kernel\(((?:[^()]|\([^()]*\))*)\)", text)
        found[os.path.basename(path)] = [c.rsplit(",", 1)[1].strip() for c in calls]
    assert {"fat_attn_fwd.cu", "fat_paged_few.cu", "fat_paged_tile.cu"} <= set(found)
    for name, needs in found.items():
        assert needs and all(re.fullmatch(r"\w*(::)?(REGS_NEEDED|kRegsNeeded)", n) for n in needs), \
            (name, needs)


@pytest.mark.parametrize("d,hq,hkv", [(64, 12, 12), (128, 16, 4), (64, 32, 1), (128, 8, 8)])
def test_workspace_size_never_falls_with_the_bounds(lib, d, hq, hkv):
    """A buffer for the largest step serves every smaller one: the size for a call is at most what any
    call of larger bounds is told."""
    c = _cache(num_heads=hkv, head_dim=d, stride_head=d, stride_token=hkv * d,
               stride_page=16 * hkv * d)

    def size(total_q, n, max_q, max_k):
        return lib.fat_paged_attn_workspace_size(
            fa._PagedShape(total_q, n, max_q, max_k, hq, 1 << 20, None), ctypes.byref(c))

    keys = (1, 380, 400, 760, 770, 1000, 1024, 1025, 4096, 100000)
    queries = (1, 2, 4, 5, 16, 17, 512)
    for n in (1, 4, 40):
        for i, k in enumerate(keys):
            for j, q in enumerate(queries):
                for total in (1, n * q - 1, n * q, n * q + 7):
                    if total < 1:
                        continue
                    s = size(total, n, q, k)
                    for t2, n2, q2, k2 in ((total + 1, n, q, k), (n * q, n, q, k),
                                           (total, n + 1, q, k),
                                           (total, n, queries[min(j + 1, len(queries) - 1)], k),
                                           (total, n, q, keys[min(i + 1, len(keys) - 1)]),
                                           (n * 512, n, 512, k), (n * 512, n, 512, 100000)):
                        if t2 >= total and q2 >= q and k2 >= k:
                            assert size(t2, n2, q2, k2) >= s, (total, n, q, k, t2, n2, q2, k2)


def _plan_places():
    """Places (from FAKE on, in entries) of the nine arrays of _plan, in its order, side by side."""
    sizes = [2, 2, 3, 8, 3, 2, 5, 5, 2]  # ctx, new, free, table, cu, lens, positions, slots, counts
    places = [sum(sizes[:i]) for i in range(9)]
    return sizes, places


@pytest.mark.parametrize("out", [3, 4, 5, 6, 7, 8])
def test_plan_results_over_other_arrays_are_refused(lib, out):
    """Lengths updated in place (seqlens_k over ctx_lens), say: other blocks still read them."""
    sizes, places = _plan_places()
    for other in range(9):
        if other == out:
            continue
        for at in (places[other], places[other] + sizes[other] - 1, places[other] + 1 - sizes[out]):
            p = [FAKE + 4 * (x + 64) for x in places]
            # the other arrays lie far away, so that these two alone overlap
            p = [x + (1 << 16) * i if i not in (out, other) else x for i, x in enumerate(p)]
            p[out] = FAKE + 4 * (at + 64)
            assert _plan(lib, dict(enumerate(p)), num_seqs=2) == -2, (out, other, at)


@pytest.mark.parametrize("kw", [dict(factor=1e-320), dict(factor=5e-324, base=2.0),
                                dict(factor=5e-324, ramp=(1.0, 4.0, 64.0)),
                                dict(amplitude=1e-60), dict(amplitude=1e-46)])
def test_rope_init_values_that_vanish_are_refused(kw):
    """A frequency that overflows, an amplitude that is 0 in the record's fp32."""
    with pytest.raises(fa.FatAttnError) as e:
        fa.fat_rope_init(64, **kw)
    assert e.value.code == -2
    fa.fat_rope_init(64, factor=1e-3, amplitude=1e-44)  # small, but a rotation
