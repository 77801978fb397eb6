"""GPU parity of the paged-cache operators: the step's maps (exact), rotary positions and appended
rows, and attention over pages against the fp64 oracle; then a decode loop that uses them together."""
import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa
import oracle
from attention_relative_position_gb300 import workloads as wl
from oracle import paged

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a, dtype=np.int32), device=DEV)


def _bf16(rng, *shape, std=1.0):
    a = torch.from_numpy(rng.normal(0.0, std, shape).astype(np.float32))
    return a.to(torch.bfloat16).to(DEV)


def _wide(t):
    return t.float().cpu().numpy().astype(np.float64)


def _errors():
    torch.cuda.synchronize()
    return fa.fat_attn_get_device_error()


@pytest.fixture(autouse=True)
def _clean_error_word():
    _errors()


# ---- plan ---------------------------------------------------------------------------------------
def _plan_inputs(rng, n, page, width, c_hi, n_hi, spare):
    ctx = rng.integers(0, c_hi + 1, n)
    new = rng.integers(0, n_hi + 1, n)
    have, want = -(-ctx // page), -(-(ctx + new) // page)
    order = rng.permutation(int(want.sum()) + spare)
    table = np.full((n, width), -7, np.int64)
    at = 0
    for i in range(n):
        table[i, :have[i]] = order[at:at + have[i]]
        at += have[i]
    return ctx, new, order[at:], table, len(order)


def _check_plan(ctx, new, free, table, page, pages, max_tokens, bits=0):
    want = paged.plan(ctx, new, free, table, page, pages, max_tokens)
    t = _i32(table)
    got = fa.fat_paged_plan(_i32(ctx), _i32(new), _i32(free), t, page, pages, max_tokens)
    assert _errors() == bits
    for name, g, w in zip(("table", "cu", "lk", "pos", "slots", "counts"), (t,) + got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


@pytest.mark.parametrize("n,page,c_hi,n_hi,pad", [
    (1, 16, 0, 1, 0), (1, 64, 500, 700, 3), (3, 16, 40, 5, 0), (64, 16, 1000, 1, 7),
    (1023, 32, 300, 40, 0), (1024, 16, 100, 1, 1), (1025, 64, 64, 70, 100), (5000, 16, 90, 3, 5)])
def test_plan(n, page, c_hi, n_hi, pad):
    rng = np.random.default_rng(n + page)
    width = -(-(c_hi + n_hi) // page)
    ctx, new, free, table, pages = _plan_inputs(rng, n, page, width, c_hi, n_hi, 9)
    _check_plan(ctx, new, free, table, page, pages, int(new.sum()) + pad)


def test_plan_shortages_and_bad_lengths():
    rng = np.random.default_rng(5)
    ctx, new, free, table, pages = _plan_inputs(rng, 40, 16, 12, 100, 60, 0)
    total = int(new.sum())
    # the free list ends early: -1 pages and slots from there on
    _check_plan(ctx, new, free[:len(free) // 2], table, 16, pages, total, fa.FAT_DEVERR_PAGES)
    # a request that its table row does not hold takes no pages
    ctx2 = ctx.copy()
    ctx2[7] = 12 * 16 + 1
    _check_plan(ctx2, new, free, table, 16, pages, total, fa.FAT_DEVERR_PAGES)
    # indexes outside the pool, in the table (a page that is continued) and in the free list
    ctx3, new3, tab3, free3 = ctx.copy(), new.copy(), table.copy(), free.copy()
    ctx3[3], new3[3], tab3[3, 0] = 5, 4, pages + 1
    free3[2] = -5
    _check_plan(ctx3, new3, free3, tab3, 16, pages, int(new3.sum()), fa.FAT_DEVERR_PAGES)
    # negative lengths count as none; more tokens than the arrays hold
    ctx4, new4 = ctx.copy(), new.copy()
    ctx4[2], new4[9] = -1, -5
    _check_plan(ctx4, new4, free, table, 16, pages, total, fa.FAT_DEVERR_SEQLENS)
    _check_plan(ctx, new, free, table, 16, pages, total - 50, fa.FAT_DEVERR_SEQLENS)


def test_plan_empty():
    t = torch.empty((0, 4), dtype=torch.int32, device=DEV)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    cu, lk, pos, slots, counts = fa.fat_paged_plan(e, e, e, t, 16, 4, 3)
    assert _errors() == 0
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3
    assert counts.tolist() == [0, 0]


# ---- rotary positions ---------------------------------------------------------------------------
# One bf16 rounding of the exact rotation (at most half a step, 2^-8 of the value) plus the fp32
# arithmetic: the angle is cut to 2^-24 turns (2 pi 2^-24 = 3.8e-7 rad), cosine and sine carry two
# fp32 roundings and the amplitude one, the two products and the sum three more, each 2^-24 of the
# pair's norm r: (3.8e-7 + 6 * 2^-24) r < 1e-6 r.
def _check_rope(got, exact, x, rot, amplitude, interleaved):
    h = rot // 2
    first = np.arange(0, rot, 2) if interleaved else np.arange(h)
    second = first + (1 if interleaved else h)
    tol = 2.0 ** -8 * np.abs(exact)
    r = amplitude * np.hypot(x[..., first], x[..., second])
    tol[..., first] += 1e-6 * r
    tol[..., second] += 1e-6 * r
    assert (np.abs(got - exact) <= tol).all()
    np.testing.assert_array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("T,H,d,rot,inter,kw", [
    (1, 1, 64, 64, True, {}), (5, 3, 128, 64, False, {}), (300, 7, 64, 16, True, dict(factor=4.0)),
    (33, 40, 128, 128, False, dict(base=500000.0, factor=8.0, ramp=(1.0, 4.0, 8192.0))),
    (2500, 2, 96, 48, False, dict(amplitude=1.25)), (700, 5, 256, 256, True, {}),
    (17, 4, 80, 32, True, dict(base=100.0))])
def test_rope_embed(T, H, d, rot, inter, kw):
    rng = np.random.default_rng(T + d)
    wide = _bf16(rng, T, H + 3, d)
    pos = rng.integers(0, 1 << 20, T)
    pos[:1] = 0
    pos[-1:] = rng.integers(0, 100)
    rope = fa.fat_rope_init(rot, interleaved=inter, **kw)
    okw = {k: v for k, v in kw.items()}
    amp = okw.get("amplitude", 1.0)
    for x in (wide[:, 1:1 + H], wide[:, :H].contiguous()):
        xin = _wide(x)
        for inverse in (False, True):
            got = fa.fat_rope_embed(x, _i32(pos), rope, inverse=inverse)
            exact = paged.rope(xin, pos, rot, interleaved=inter, inverse=inverse, **okw)
            _check_rope(_wide(got), exact, xin, rot, amp, inter)
    y = wide.clone()  # in place, inside a larger array: the other heads stay
    fa.fat_rope_embed(y[:, 2:2 + H], _i32(pos), rope, out=y[:, 2:2 + H])
    _check_rope(_wide(y[:, 2:2 + H]), paged.rope(_wide(wide[:, 2:2 + H]), pos, rot,
                                                 interleaved=inter, **okw),
                _wide(wide[:, 2:2 + H]), rot, amp, inter)
    assert torch.equal(y[:, :2], wide[:, :2]) and torch.equal(y[:, 2 + H:], wide[:, 2 + H:])
    assert _errors() == 0


def test_rope_embed_far_negative_and_repeated_rows():
    rng = np.random.default_rng(8)
    pos = np.array([2 ** 31 - 1, -1, -12345, 2 ** 31 - 1, 7])
    x = _bf16(rng, 1, 2, 64).expand(5, 2, 64)  # one row for every position
    rope = fa.fat_rope_init(64)
    got = _wide(fa.fat_rope_embed(x, _i32(pos), rope))
    # the angle in whole turns by rational arithmetic: 64-bit floats lose it at 2^31
    from fractions import Fraction
    import math
    rate = [Fraction(r, 1 << 64) for r in rope.rate[:32]]
    turn = np.array([[float((int(p) * r) % 1) for r in rate] for p in pos]) * 2 * math.pi
    xin = _wide(x)
    u, v = xin[..., 0::2], xin[..., 1::2]
    exact = np.empty_like(xin)
    exact[..., 0::2] = u * np.cos(turn)[:, None] - v * np.sin(turn)[:, None]
    exact[..., 1::2] = u * np.sin(turn)[:, None] + v * np.cos(turn)[:, None]
    _check_rope(got, exact, xin, 64, 1.0, True)


def test_rope_equals_document_rope():
    """Positions counted in each document, interleaved, whole head: fat_rope_apply bit for bit."""
    w = wl.Workload("rope_pair", (300, 1, 77), 3, 128, 1.0, seed=91)
    x = wl.make_inputs(w, device=DEV)
    pos = np.concatenate([np.arange(n) for n in (300, 1, 77)])
    a = fa.fat_rope_apply(x["q"], x["cu_seqlens"], w.max_seqlen)
    b = fa.fat_rope_embed(x["q"], _i32(pos), fa.fat_rope_init(128))
    assert torch.equal(a, b)


# ---- append -------------------------------------------------------------------------------------
def _make_cache(pages, page, H, d, layout, fill):
    """(k, v) views [pages, page, H, d] of one of the memory layouts a program may keep."""
    if layout == "token":
        k, v = (torch.full((pages, page, H, d), fill, dtype=torch.bfloat16, device=DEV)
                for _ in range(2))
    elif layout == "head":  # heads outside the tokens of a page
        k, v = (torch.full((pages, H, page, d), fill, dtype=torch.bfloat16,
                           device=DEV).transpose(1, 2) for _ in range(2))
    else:  # keys and values of a page in one block
        both = torch.full((pages, 2, page, H, d), fill, dtype=torch.bfloat16, device=DEV)
        k, v = both[:, 0], both[:, 1]
    return k, v


@pytest.mark.parametrize("layout", ["token", "head", "block"])
@pytest.mark.parametrize("T,hq,hkv,d,rot,inter", [(1, 1, 1, 64, 64, True), (37, 6, 2, 128, 64, False),
                                                  (900, 4, 4, 64, 32, True), (5, 3, 3, 96, 0, True)])
def test_append(layout, T, hq, hkv, d, rot, inter):
    rng = np.random.default_rng(T)
    page, pages = 16, 2 * (T // 16 + 2)
    qkv = _bf16(rng, T, hq + 2 * hkv, d)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    slots = rng.permutation(pages * page)[:T]
    if T > 4:
        slots[2] = -1  # padding
    pos = rng.integers(0, 100000, T)
    kc, vc = _make_cache(pages, page, hkv, d, layout, 7.0)
    rope = fa.fat_rope_init(rot, interleaved=inter) if rot else None
    qo = fa.fat_paged_append(k, v, kc, vc, _i32(slots), q=q, positions=_i32(pos), rope=rope)
    assert _errors() == 0
    want_v = np.full((pages * page, hkv, d), 7.0)
    kx = paged.rope(_wide(k), pos, rot, interleaved=inter) if rot else _wide(k)
    qx = paged.rope(_wide(q), pos, rot, interleaved=inter) if rot else _wide(q)
    ok = slots >= 0
    want_v[slots[ok]] = _wide(v)[ok]
    np.testing.assert_array_equal(_wide(vc).reshape(-1, hkv, d), want_v)
    got_k = _wide(kc).reshape(-1, hkv, d)
    other = np.ones(pages * page, bool)
    other[slots[ok]] = False
    assert (got_k[other] == 7.0).all()
    _check_rope(got_k[slots[ok]], kx[ok], _wide(k)[ok], rot, 1.0, inter)
    _check_rope(_wide(qo), qx, _wide(q), rot, 1.0, inter)
    # without queries: the same rows
    kc2, vc2 = _make_cache(pages, page, hkv, d, layout, 7.0)
    assert fa.fat_paged_append(k, v, kc2, vc2, _i32(slots), positions=_i32(pos), rope=rope) is None
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_append_slot_outside_is_dropped_and_reported():
    rng = np.random.default_rng(3)
    k = _bf16(rng, 3, 2, 64)
    kc, vc = _make_cache(4, 16, 2, 64, "token", 0.0)
    fa.fat_paged_append(k, k, kc, vc, _i32([63, 64, 2 ** 31 - 1]))
    assert _errors() == fa.FAT_DEVERR_INDEX
    assert torch.equal(kc.view(-1, 2, 64)[63], k[0]) and (kc.view(-1, 2, 64)[:63] == 0).all()


# ---- attention ----------------------------------------------------------------------------------
class Problem:
    """Requests with queries, contexts and pages; stale slots and unused pages hold `stale`."""

    def __init__(self, lq, lk, hq, hkv, d, page, t5=None, alibi=False, causal=True, seed=0,
                 layout="token", stale=float("nan"), std=1.0, scale=None, pad=0):
        rng = np.random.default_rng(seed)
        self.lq, self.lk = np.array(lq), np.array(lk)
        self.n, self.hq, self.hkv, self.d, self.page = len(lq), hq, hkv, d, page
        self.scale = d ** -0.5 if scale is None else scale
        self.causal, self.t5 = causal, t5
        used = -(-self.lk // page)
        self.pages = int(used.sum()) + 3
        self.width = max(1, int(used.max()) if self.n else 1)
        order = rng.permutation(self.pages)
        self.kc, self.vc = _make_cache(self.pages, page, hkv, d, layout, stale)
        self.table = np.full((self.n, self.width), 1 << 30)  # entries behind a request: unread
        at = 0
        for i in range(self.n):
            mine = order[at:at + used[i]]
            at += used[i]
            self.table[i, :used[i]] = mine
            m = int(self.lk[i])
            if m:
                sl = torch.as_tensor(np.repeat(mine, page)[:m] * page + np.arange(m) % page)
                pg, off = (sl // page).to(DEV), (sl % page).to(DEV)
                self.kc[pg, off] = _bf16(rng, m, hkv, d, std=std)
                self.vc[pg, off] = _bf16(rng, m, hkv, d)
        self.cu = np.concatenate([[0], np.cumsum(self.lq)])
        self.total = int(self.cu[-1])
        self.q = _bf16(rng, self.total + pad, hq, d, std=std)
        self.bias = self.slopes = None
        if t5:
            self.bias = torch.from_numpy(rng.normal(0, 0.5, (t5[0], hq)).astype(np.float32)).to(DEV)
        if alibi:
            self.slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float().to(DEV)

    def kwargs(self):
        t5 = self.t5 or (0, 0, True)
        return dict(bias_table=self.bias, num_buckets=t5[0], max_distance=t5[1],
                    bidirectional=t5[2], alibi_slopes=self.slopes, causal=self.causal,
                    softmax_scale=self.scale)

    def arrays(self):
        return _i32(self.table), _i32(self.cu), _i32(self.lk)

    def run(self, arrays=None, **kw):
        args = dict(max_q=int(max(self.lq, default=0)), max_k=int(max(self.lk, default=0)))
        args.update({k: kw.pop(k) for k in ("max_q", "max_k") if k in kw})
        return fa.fat_paged_attn(self.q, self.kc, self.vc, *(arrays or self.arrays()),
                                 args["max_q"], args["max_k"], **self.kwargs(), **kw)

    def oracle(self):
        t5 = self.t5 or (0, 0, True)
        return paged.attention(
            _wide(self.q), _wide(self.kc), _wide(self.vc), self.table, self.cu, self.lk,
            table=None if self.bias is None else _wide(self.bias), num_buckets=t5[0],
            max_distance=t5[1], bidirectional=t5[2],
            slopes=None if self.slopes is None else _wide(self.slopes), causal=self.causal,
            scale=self.scale)

    def check(self, out, lse, rows=None):
        """Tolerances. A logit x (of size S + B at most) is formed in fp32: d products summed
        (d 2^-24 S), scaled, and the bias added (4 2^-24 (S + B)): ex. Every weight then carries
        ex + 2^-20 (the exponential) relative, before it is rounded to bf16 (2^-8) as an operand of
        P V and normalised by the sum of the unrounded weights; the output is rounded once more."""
        ro, rl, a, s, b = self.oracle()
        ex = (self.d * s + 4 * (s + b)) * 2.0 ** -24
        got, gl = _wide(out[:self.total]), lse.cpu().numpy()[:, :self.total].astype(np.float64)
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
    "one_token": dict(lq=[1], lk=[1], hq=1, hkv=1, d=64, page=16),
    "no_keys": dict(lq=[1, 2, 1], lk=[0, 0, 5], hq=4, hkv=2, d=128, page=16, causal=False),
    "page_edges": dict(lq=[1] * 9, lk=[15, 16, 17, 31, 32, 33, 63, 64, 65], hq=2, hkv=2, d=64,
                       page=16, t5=T5D),
    "tile_edges_d128": dict(lq=[1] * 7, lk=[127, 128, 129, 255, 256, 257, 300], hq=8, hkv=2, d=128,
                            page=64, alibi=True),
    "decode_t5_ragged": dict(lq=[1] * 12, lk=[1, 2, 3000, 700, 64, 65, 900, 1, 128, 1500, 33, 500],
                             hq=12, hkv=12, d=64, page=32, t5=T5D, scale=1.0, std=0.4),
    "decode_gqa16": dict(lq=[1] * 5, lk=[4000, 17, 800, 0, 129], hq=32, hkv=2, d=128, page=16),
    "decode_gqa3_bidir": dict(lq=[1, 1, 0, 1], lk=[900, 40, 30, 2222], hq=9, hkv=3, d=64,
                              page=256, t5=T5B, causal=False),
    "draft_group4": dict(lq=[4, 3, 1, 2, 0, 4], lk=[1200, 3, 9, 130, 7, 4], hq=8, hkv=2, d=128,
                         page=16, t5=T5D, alibi=True),
    "draft_fewer_keys": dict(lq=[5, 7, 3], lk=[2, 7, 0], hq=4, hkv=4, d=64, page=16, alibi=True),
    "chunk_group1": dict(lq=[200, 1, 130], lk=[700, 400, 130], hq=2, hkv=2, d=64, page=32, t5=T5D),
    "chunk_group5_d128": dict(lq=[70, 33, 1, 129], lk=[300, 33, 900, 129], hq=10, hkv=2, d=128,
                              page=16, alibi=True),
    "chunk_group3_bidir": dict(lq=[100, 260], lk=[1000, 300], hq=3, hkv=1, d=64, page=128, t5=T5B,
                               alibi=True, causal=False),
    "chunk_fewer_keys": dict(lq=[300, 140, 260], lk=[100, 0, 130], hq=4, hkv=2, d=128, page=64),
    "chunk_group8_long": dict(lq=[40, 300], lk=[5000, 2600], hq=16, hkv=2, d=128, page=64,
                              alibi=True),
    "chunk_group16": dict(lq=[64, 17], lk=[64, 1000], hq=16, hkv=1, d=64, page=16),
    "chunk_group128": dict(lq=[3, 1], lk=[200, 77], hq=128, hkv=1, d=64, page=16, t5=T5D),
    "chunk_group100": dict(lq=[5], lk=[300], hq=100, hkv=1, d=128, page=32),
    "mixed": dict(lq=[1, 1, 250, 1, 3, 1, 40], lk=[2000, 30, 1000, 1, 800, 0, 41], hq=8, hkv=2,
                  d=64, page=16, t5=T5D),
    "mixed_d128": dict(lq=[1, 300, 1, 1], lk=[3000 - 1, 420, 64, 8], hq=4, hkv=4, d=128, page=256),
    "many_requests": dict(lq=[1] * 700, lk=list(np.random.default_rng(1).integers(1, 60, 700)),
                          hq=2, hkv=1, d=64, page=16, t5=T5D),
    "many_chunks": dict(lq=list(np.random.default_rng(2).integers(0, 30, 500)),
                        lk=list(np.random.default_rng(3).integers(30, 90, 500)), hq=4, hkv=2, d=64,
                        page=16),
    "decode_many": dict(lq=[1] * 700, lk=list(np.random.default_rng(4).integers(0, 90, 700)), hq=4,
                        hkv=4, d=64, page=16, t5=T5D),
    "million_keys": dict(lq=[1, 1], lk=[1 << 20, 900001], hq=2, hkv=1, d=64, page=256, t5=T5D),
    "chunk_long_context": dict(lq=[20], lk=[300007], hq=2, hkv=2, d=128, page=4096, alibi=True),
    # logits of hundreds: the running reference moves by more than 2^32 and 2^64, in either half of a
    # key tile, after rows without a key and with grouped heads
    "large_logits_d128": dict(lq=[150, 40, 300], lk=[900, 500, 250], hq=4, hkv=2, d=128, page=16,
                              std=3.0, scale=1.0),
    "large_logits_alibi_d128": dict(lq=[130], lk=[1400], hq=3, hkv=3, d=128, page=64, alibi=True,
                                    std=4.0, scale=1.0, causal=False),
    "large_logits": dict(lq=[1, 150], lk=[500, 400], hq=2, hkv=2, d=64, page=16, t5=T5D, std=3.0,
                         scale=1.0),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    p = Problem(seed=sum(map(ord, name)), **CASES[name])
    out, lse = p.run()
    assert _errors() == 0
    p.check(out, lse)


FINE_CASES = {
    "whole_d64": dict(lq=[1] * 4, lk=[2, 7, 40, 500], hq=12, hkv=12, d=64, page=16, t5=T5D),
    "whole_d128": dict(lq=[1] * 5, lk=[3, 16, 17, 200, 380], hq=16, hkv=2, d=128, page=16),
    "cut_d64": dict(lq=[1, 5, 2], lk=[3000, 1500, 9], hq=6, hkv=2, d=64, page=32, alibi=True),
    "cut_d128": dict(lq=[1, 4, 2], lk=[4000, 33, 700], hq=8, hkv=2, d=128, page=64, causal=False),
    "beside_chunk": dict(lq=[1, 1, 60], lk=[600, 12, 90], hq=8, hkv=2, d=64, page=16),
    "beside_chunk_d128": dict(lq=[1, 3, 70], lk=[2000, 5, 90], hq=4, hkv=2, d=128, page=16),
}


@pytest.mark.parametrize("name", FINE_CASES)
def test_attention_of_few_rows_keeps_its_weights(name):
    """At most 16 rows: the weights enter P V with 16 bits, as those of the decode kernel over packed
    keys do with 24, so only the output's own rounding is of bf16 size. Tolerance: 2^-8 of the value;
    per |weight x value| twice the logits' ex (as in check), 2^-20 of the exponential, 2^-17 of the
    weight's two parts, and the fp32 accumulation, a key block of 16 at a time and twice (for both
    parts): lk / 8 additions that each lose 2^-22 of the sum so far at most."""
    p = Problem(seed=70, **FINE_CASES[name])
    out, _ = p.run()
    assert _errors() == 0
    ro, _, a, s, b = p.oracle()
    group = p.hq // p.hkv
    for i in range(p.n):
        if p.lq[i] * group > 16:
            continue
        rows = slice(int(p.cu[i]), int(p.cu[i + 1]))
        ex = (p.d * s + 4 * (s + b)) * 2.0 ** -24
        fine = 2 * ex + 2.0 ** -20 + 2.0 ** -17 + (p.lk[i] / 8 + 2) * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(ro[rows]) + fine * a[rows] + 1e-30
        err = np.abs(_wide(out[rows]) - ro[rows])
        assert (err <= tol).all(), (i, (err / tol).max())


@pytest.mark.parametrize("layout", ["head", "block"])
@pytest.mark.parametrize("name", ["decode_gqa16", "chunk_group5_d128", "mixed"])
def test_attention_cache_layouts(layout, name):
    """The memory layout of the cache changes nothing: bit for bit the token-major result."""
    a = Problem(seed=11, **CASES[name])
    b = Problem(seed=11, layout=layout, **CASES[name])
    oa, la = a.run()
    ob, lb = b.run()
    assert _errors() == 0
    assert torch.equal(oa, ob) and torch.equal(la, lb)


def test_cache_of_one_page_inside_a_block_of_layers():
    """A single page whose heads lie outside its tokens, two layers apart: appended and attended to as
    the same page on its own."""
    rng = np.random.default_rng(12)
    S, H, d = 32, 2, 64
    k, v, q = _bf16(rng, 20, H, d), _bf16(rng, 20, H, d), _bf16(rng, 3, H, d)
    block = torch.full((2, H, 2, S, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    alone = torch.full((2, 1, S, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    got = []
    for kc, vc in ((block[0, :, 1].transpose(0, 1)[None], block[1, :, 1].transpose(0, 1)[None]),
                   (alone[0], alone[1])):
        fa.fat_paged_append(k, v, kc, vc, _i32(range(20)))
        got.append(fa.fat_paged_attn(q, kc, vc, _i32([[0]]), _i32([0, 3]), _i32([20]), 3, 20,
                                     causal=True, softmax_scale=0.125))
    assert _errors() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all()
    assert block[:, :, 0].isnan().all() and block[:, :, 1, 20:].isnan().all()


@pytest.mark.parametrize("pages,H", [(1, 2), (3, 1), (1, 1)])
def test_caches_whose_single_entries_have_other_strides(pages, H):
    """Keys cut out of a larger block, values on their own: strides over a single page or head differ
    and say nothing."""
    rng = np.random.default_rng(13)
    S, d, n = 16, 64, 16 * pages
    k, v, q = _bf16(rng, n, H, d), _bf16(rng, n, H, d), _bf16(rng, 2, H, d)
    if pages == 1:
        kc = torch.full((4, 2, S, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)[2:3, 1]
    else:  # one head, as a view that has a stride of its own for it
        kc = torch.full((pages, S, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
        kc = kc.as_strided(kc.shape, (S * d, d, 8, 1))
    vc = torch.full((pages, S, H, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert kc.stride() != vc.stride()
    k2, v2 = kc.clone(memory_format=torch.contiguous_format), vc.clone()
    got = []
    for a, b in ((kc, vc), (k2, v2)):
        fa.fat_paged_append(k, v, a, b, _i32(range(n)))
        got.append(fa.fat_paged_attn(q, a, b, _i32([list(range(pages))]), _i32([0, 2]), _i32([n]), 2, n,
                                     causal=True, softmax_scale=0.125))
    assert _errors() == 0
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert got[0][0].isfinite().all()


@pytest.mark.parametrize("stale", [float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("name", ["decode_t5_ragged", "chunk_group1", "mixed_d128"])
def test_attention_ignores_stale_slots(stale, name):
    a, b = Problem(seed=4, **CASES[name]), Problem(seed=4, stale=stale, **CASES[name])
    oa, la = a.run()
    ob, lb = b.run()
    assert torch.equal(oa, ob) and torch.equal(la, lb)


@pytest.mark.parametrize("name", ["decode_gqa16", "mixed", "chunk_group8_long"])
def test_attention_bounds_padding_and_repeats(name):
    """Loose bounds, rows behind the last request, given outputs, a second run of the same call."""
    p = Problem(seed=5, pad=19, **CASES[name])
    a, la = p.run()
    out = torch.full_like(p.q, 3.0)
    lse = torch.full((p.hq, p.q.shape[0]), 5.0, device=DEV)
    size = fa.fat_paged_attn_workspace_size(p.q, p.kc, _i32(p.cu), 4 * max(p.lq), 8 * max(p.lk))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    p.run(out=out, lse=lse, workspace=ws, max_q=4 * int(max(p.lq)), max_k=8 * int(max(p.lk)))
    assert _errors() == 0
    assert (out[p.total:] == 3.0).all() and (lse[:, p.total:] == 5.0).all()
    p.check(out, lse)
    p.check(a, la)
    b, lb = p.run()
    assert torch.equal(a[:p.total], b[:p.total]) and torch.equal(la[:, :p.total], lb[:, :p.total])


@pytest.mark.parametrize("hq,hkv,d", [(16, 4, 128), (6, 2, 64)])
def test_one_workspace_serves_every_smaller_step(hq, hkv, d):
    """A buffer for the largest bounds: a chunk, a full batch of equal chunks, the same with padding and
    single tokens run in it."""
    small = dict(hq=hq, hkv=hkv, d=d, page=16, alibi=True)
    for lk in (1000, 3000):
        steps = [Problem(lq=[200, 30, 1, 1], lk=[lk, 700, 900, 40], seed=80, **small),
                 Problem(lq=[50] * 4, lk=[lk, 700, 900, 50], seed=81, **small),
                 Problem(lq=[50, 50, 50, 49], lk=[lk, 700, 900, 50], seed=82, **small),
                 Problem(lq=[1] * 4, lk=[lk, 700, 900, 40], seed=83, **small),
                 Problem(lq=[2, 1], lk=[lk, 600], seed=84, **small)]
        big = steps[0]
        size = fa.fat_paged_attn_workspace_size(big.q, big.kc, _i32(big.cu), 200, lk)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        for p in steps:
            assert p.total <= big.total and p.n <= big.n
            out, lse = p.run(workspace=ws, max_q=int(max(p.lq)))
            assert _errors() == 0
            p.check(out, lse)


@pytest.mark.parametrize("d,lq", [(64, [1] * 6), (128, [2] * 6), (64, [40, 1, 90, 3, 1, 33]),
                                  (128, [70] * 6)])
def test_requests_share_pages(d, lq):
    """A common prefix of whole pages, named by every request: bit for bit the results over copies."""
    page, prefix = 16, 1600
    lk = [prefix + n + 7 * i for i, n in enumerate(lq)]
    p = Problem(lq=lq, lk=lk, hq=8, hkv=2, d=d, page=page, alibi=True, seed=90)
    m = prefix // page
    for i in range(1, p.n):  # the first request's prefix, copied into the others' pages
        for c in (p.kc, p.vc):
            c[torch.as_tensor(p.table[i, :m])] = c[torch.as_tensor(p.table[0, :m])]
    want, wl = p.run()
    for i in range(1, p.n):
        for c in (p.kc, p.vc):
            c[torch.as_tensor(p.table[i, :m])] = float("nan")  # read no more
        p.table[i, :m] = p.table[0, :m]
    out, lse = p.run()
    assert _errors() == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)
    p.check(out, lse)


@pytest.mark.parametrize("lq,pad", [([40, 1, 3, 40], 76), ([9, 9, 9], 0), ([1, 0, 0, 33], 98)])
def test_attention_rows_that_look_equal(lq, pad):
    """total_q = num_seqs * max_seqlen_q, with equal requests or with padding: every row is there."""
    p = Problem(lq=lq, lk=[1500, 64, 2000, 70][:len(lq)], hq=4, hkv=2, d=64, page=16, pad=pad,
                alibi=True, seed=40)
    assert p.q.shape[0] == len(lq) * max(lq)
    out = torch.full_like(p.q, 3.0)
    _, lse = p.run(out=out)
    assert _errors() == 0
    p.check(out, lse)
    assert (out[p.total:] == 3.0).all()


@pytest.mark.parametrize("name", ["decode_gqa16", "chunk_group5_d128", "chunk_group1"])
@pytest.mark.parametrize("bad", [-1, 1 << 20, -(1 << 31)])
def test_attention_bad_page_counts_as_zeros(name, bad):
    p = Problem(seed=6, **CASES[name])
    p.table[0, 0] = bad
    out, lse = p.run()
    assert _errors() == fa.FAT_DEVERR_PAGES
    p.check(out, lse)


@pytest.mark.parametrize("lq", [[1, 1, 2], [40, 3]])
def test_attention_without_any_key(lq):
    """No request has a key yet: an empty block table, bounds of 0; rows of zeros."""
    p = Problem(lq=lq, lk=[0] * len(lq), hq=4, hkv=2, d=64, page=16, causal=False, pad=2)
    out = torch.full_like(p.q, 3.0)
    _, lse = fa.fat_paged_attn(
        p.q, p.kc, p.vc, torch.empty((p.n, 0), dtype=torch.int32, device=DEV), _i32(p.cu),
        _i32(p.lk), max(lq), 0, out=out, **p.kwargs())
    assert _errors() == 0
    assert (out[:p.total] == 0).all() and (out[p.total:] == 3.0).all()
    assert (lse[:, :p.total] == -float("inf")).all()


NAN_CASES = {
    "decode_whole": dict(lq=[1, 1, 1], lk=[40, 700, 64], hq=4, hkv=2, d=64, page=16),
    "decode_cut_d128": dict(lq=[1, 4], lk=[30000, 9000], hq=8, hkv=2, d=128, page=64, alibi=True),
    "chunk_d64": dict(lq=[200, 40], lk=[5000, 41], hq=4, hkv=4, d=64, page=32),
    "chunk_cut_d128": dict(lq=[150, 60], lk=[6000, 700], hq=4, hkv=2, d=128, page=16),
}


@pytest.mark.parametrize("name", NAN_CASES)
def test_attention_nan_queries_and_keys_show(name):
    """A NaN query leaves its own row NaN, a NaN key every row that sees it; no other row changes."""
    p = Problem(seed=51, **NAN_CASES[name])
    want, wl = p.run()
    row, h = p.total - 1, 1
    p.q[row, h, 5] = float("nan")
    out, lse = p.run()
    assert out[row, h].isnan().all() and lse[h, row].isnan()
    keep = torch.ones(p.total, p.hq, dtype=torch.bool, device=DEV)
    keep[row, h] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse.t()[keep], wl.t()[keep])
    p = Problem(seed=51, **NAN_CASES[name])
    key = int(p.lk[0]) - int(p.lq[0])  # the first query's own position: every query sees it
    p.kc[int(p.table[0, key // p.page]), key % p.page, 0, 9] = float("nan")
    out, lse = p.run()
    group, n = p.hq // p.hkv, int(p.lq[0])
    assert out[:n, :group].isnan().all() and lse[:group, :n].isnan().all()
    keep = torch.ones(p.total, p.hq, dtype=torch.bool, device=DEV)
    keep[:n, :group] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse.t()[keep], wl.t()[keep])
    assert _errors() == 0


@pytest.mark.parametrize("low", [-float("inf"), float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("case", [
    dict(lq=[1, 1, 3], lk=[900, 5, 3000], hq=4, hkv=2, d=64, page=16, t5=T5D, alibi=True),
    dict(lq=[1] * 3, lk=[2000, 10, 90], hq=8, hkv=2, d=128, page=16, t5=T5D),
    dict(lq=[130, 300], lk=[2500, 300], hq=4, hkv=2, d=64, page=16, t5=T5D),
    dict(lq=[130, 300], lk=[2500, 300], hq=4, hkv=2, d=128, page=16, t5=T5B, causal=False),
], ids=["few_d64", "few_d128", "tile_d64", "tile_d128"])
def test_attention_bias_that_masks(case, low):
    """Table entries of -infinity (or the type's lowest value): their keys are masked; a head with
    nothing else has no keys at all. The oracle gets -1e6 instead, whose weights are exactly 0
    beside any other key; rows of such keys alone are told by their lse. Tolerances as in check."""
    p = Problem(seed=52, **case)
    p.bias[3] = -1e6          # near keys
    p.bias[-1, 1] = -1e6      # the far side, one head
    p.bias[:, 2] = -1e6       # a head without a key
    ro, rl, a, s, _ = p.oracle()
    b = float(p.bias[p.bias > -1e5].abs().max())
    if p.slopes is not None:
        b += float(p.slopes.max()) * 3100
    p.bias[p.bias == -1e6] = low
    out, lse = p.run()
    assert _errors() == 0
    got, gl = _wide(out), lse.cpu().numpy().astype(np.float64)
    none = rl < -1e5
    assert none[2].all() and not none[0].any()
    assert (gl[none] == -np.inf).all() and (got.transpose(1, 0, 2)[none] == 0).all()
    ex = (p.d * s + 4 * (s + b)) * 2.0 ** -24
    keep = ~none.T
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 2 * ex + 2.0 ** -18) * a * 1.01 + 1e-30
    assert (np.abs(got - ro)[keep] <= tol[keep]).all()
    ltol = ex + 2.0 ** -18 + 2.0 ** -22 * np.abs(rl[~none])
    assert (np.abs(gl[~none] - rl[~none]) <= ltol).all()


def test_attention_corrupt_lengths_leave_their_rows():
    for name in ("decode_t5_ragged", "mixed", "chunk_group5_d128"):
        for what in ("long", "negative", "bound", "queries"):
            p = Problem(seed=7, **CASES[name])
            lk, cu = p.lk.copy(), p.cu.copy()
            kw = {}
            if what == "long":
                lk[0] = p.width * p.page + 1
                kw["max_k"] = 1 << 20
            elif what == "negative":
                lk[0] = -3
            elif what == "bound":
                kw["max_k"] = int(max(p.lk)) - 1
            else:
                kw["max_q"] = int(max(p.lq)) - 1
            bad = {"bound": int(np.argmax(p.lk)), "queries": int(np.argmax(p.lq))}.get(what, 0)
            skip = set()
            if what == "queries":
                if max(p.lq) == 1:
                    continue
            for i in range(p.n):
                if i == bad or (what == "queries" and p.lq[i] == max(p.lq)) or \
                        (what == "bound" and p.lk[i] == max(p.lk)):
                    skip.update(range(cu[i], cu[i + 1]))
            out = torch.full_like(p.q, 3.0)
            kwargs = dict(p.kwargs(), out=out)
            _, lse = fa.fat_paged_attn(p.q, p.kc, p.vc, _i32(p.table), _i32(cu), _i32(lk),
                                       kw.get("max_q", int(max(p.lq))),
                                       kw.get("max_k", int(max(p.lk))), **kwargs)
            assert _errors() == fa.FAT_DEVERR_SEQLENS, (name, what)
            rows = np.array([r for r in range(p.total) if r not in skip])
            gone = np.array(sorted(skip))
            assert (out[torch.as_tensor(gone)] == 3.0).all(), (name, what)
            p.check(out, lse, rows=rows)
    p = Problem(seed=7, **CASES["mixed"])
    for cu in ([0, 1, 2, 252, 253, 256, 10 ** 6, 297], [0, 1, -2, 252, 253, 256, 257, 297]):
        fa.fat_paged_attn(p.q, p.kc, p.vc, _i32(p.table), _i32(cu), _i32(p.lk), 250, 2000,
                          **p.kwargs())
        assert _errors() == fa.FAT_DEVERR_SEQLENS


def test_caches_and_rows_beyond_32_bits():
    """Caches of more than 2^32 elements and rows of more than 2^31: bit for bit the results of
    the same requests in a small cache, and of the same rows alone."""
    pages, page, hkv, d = (1 << 18) + 64, 64, 2, 128
    kc, vc = (torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device=DEV)
              for _ in range(2))
    assert kc.numel() > 1 << 32
    for name, lq, lk in (("few", [1, 2, 1], [3000, 200, 65]), ("tile", [90, 40], [1500, 41])):
        p = Problem(lq=lq, lk=lk, hq=8, hkv=hkv, d=d, page=page, seed=63)
        want, wl = p.run()
        # the small cache's pages spread over the large one, the last page among them
        to = np.linspace(pages - 1, 0, p.pages).astype(np.int64)
        kc[torch.as_tensor(to)] = p.kc
        vc[torch.as_tensor(to)] = p.vc
        table = np.where(p.table < p.pages, to[np.minimum(p.table, p.pages - 1)], 0)
        _, cu, lens = p.arrays()
        out, lse = fa.fat_paged_attn(p.q, kc, vc, _i32(table), cu, lens, int(max(lq)),
                                     int(max(lk)), **p.kwargs())
        assert torch.equal(out, want) and torch.equal(lse, wl), name
    rng = np.random.default_rng(64)
    k = _bf16(rng, 5, hkv, d)
    slots = _i32([pages * page - 1, (1 << 24) + 3, 17, pages * page - 64, 1 << 23])
    fa.fat_paged_append(k, k, kc, vc, slots)
    assert torch.equal(kc.view(-1, hkv, d)[slots.long()], k)
    assert torch.equal(vc.view(-1, hkv, d)[slots.long()], k)
    assert _errors() == 0
    del kc, vc
    x = torch.zeros((1 << 18) + 100, 64, 128, dtype=torch.bfloat16, device=DEV)
    assert x.numel() > 1 << 31
    x[-3:] = _bf16(rng, 3, 64, 128)
    pos = torch.arange(x.shape[0], dtype=torch.int32, device=DEV)
    rope = fa.fat_rope_init(128, interleaved=False)
    want = fa.fat_rope_embed(x[-3:].clone(), pos[-3:].clone(), rope)
    fa.fat_rope_embed(x, pos, rope, out=x)
    assert torch.equal(x[-3:], want) and (x[:-3] == 0).all()


def test_results_and_workspace_belong_to_the_given_stream():
    """A call on another stream than the current one: what it allocates is not handed out again
    before it has run."""
    p = Problem(seed=61, **CASES["chunk_group8_long"])
    want, wl = p.run()
    rope = fa.fat_rope_init(128)
    pos = torch.arange(p.total, dtype=torch.int32, device=DEV)
    turned = fa.fat_rope_embed(p.q, pos, rope)
    arrays = p.arrays()
    size = fa.fat_paged_attn_workspace_size(p.q, p.kc, arrays[1], int(max(p.lq)), int(max(p.lk)))
    assert size > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        out, lse = p.run(arrays=arrays, stream=side)
        y = fa.fat_rope_embed(p.q, pos, rope, stream=side)
        held = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert all((h == 7).all() for h in held)
        assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(y, turned)
        del held, out, lse, y


def test_attention_on_streams_and_from_graphs():
    """Two calls at once on their own streams and workspaces; a captured call replayed with other
    lengths, tables and queries."""
    a = Problem(seed=21, **CASES["decode_gqa16"])
    b = Problem(seed=22, **CASES["chunk_group8_long"])
    want = [x.run() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    arrays = [x.arrays() for x in (a, b)]
    outs = [dict(out=torch.empty_like(o), lse=torch.empty_like(l)) for o, l in want]
    for x, o in zip((a, b), outs):
        o["workspace"] = torch.empty(
            max(1, fa.fat_paged_attn_workspace_size(x.q, x.kc, arrays[0][1], 300, 5000)),
            dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(10):
        got = [x.run(arrays=r, stream=s, **o)
               for x, r, s, o in zip((a, b), arrays, streams, outs)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl_) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl_)
    for name, other in (("mixed", dict(lq=[3, 1, 200, 0, 1, 1, 91], lk=[500, 1, 999, 0, 64, 2, 2000])),
                        ("decode_gqa16", dict(lq=[1] * 5, lk=[1, 4000, 0, 2000, 3]))):
        p, r = Problem(seed=23, **CASES[name]), Problem(seed=24, **dict(CASES[name], **other))
        P = max(p.pages, r.pages)
        kc, vc = _make_cache(P, p.page, p.hkv, p.d, "token", 0.0)
        width = max(p.width, r.width)
        tab = torch.zeros((p.n, width), dtype=torch.int32, device=DEV)
        cu, lk = _i32(p.cu), _i32(p.lk)
        q = torch.zeros((max(p.total, r.total), p.hq, p.d), dtype=torch.bfloat16, device=DEV)
        out, lse = torch.zeros_like(q), torch.zeros((p.hq, q.shape[0]), device=DEV)

        def load(x):
            kc[:x.pages] = x.kc
            vc[:x.pages] = x.vc
            tab[:, :x.width] = _i32(np.minimum(x.table, P - 1))
            cu.copy_(_i32(x.cu))
            lk.copy_(_i32(x.lk))
            q[:x.total] = x.q

        def call():
            t5 = p.t5 or (0, 0, True)
            fa.fat_paged_attn(q, kc, vc, tab, cu, lk, 250, 4096, bias_table=p.bias,
                              num_buckets=t5[0], max_distance=t5[1], bidirectional=t5[2],
                              causal=True, softmax_scale=p.scale, out=out, lse=lse, workspace=ws)
        ws = torch.empty(max(1, fa.fat_paged_attn_workspace_size(q, kc, cu, 250, 4096)),
                         dtype=torch.uint8, device=DEV)
        load(p)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        for x in (p, r, p):
            x.bias = p.bias
            load(x)
            g.replay()
            assert _errors() == 0
            x.check(out, lse)


@pytest.mark.parametrize("name", ["decode_gqa16", "chunk_group5_d128", "mixed"])
def test_attention_watchdog(name):
    """No copies are issued: the waits run out, the status says so, and the next call is right."""
    p = Problem(seed=33, **CASES[name])
    try:
        fa.fat_attn_debug_set_watchdog(50_000_000, 1)
        p.run()
        assert _errors() == fa.FAT_DEVERR_TIMEOUT_FWD
    finally:
        fa.fat_attn_debug_set_watchdog(0, 0)
    out, lse = p.run()
    assert _errors() == 0
    p.check(out, lse)


def test_arguments_are_checked():
    p = Problem(seed=9, **CASES["decode_gqa16"])
    args = [p.q, p.kc, p.vc, _i32(p.table), _i32(p.cu), _i32(p.lk), 1, 4000]

    def refused(err, i, value):
        a = list(args)
        a[i] = value
        with pytest.raises(err):
            fa.fat_paged_attn(*a, **p.kwargs())
    refused(TypeError, 0, p.q.float())
    refused(ValueError, 0, p.q.transpose(0, 1))
    refused(ValueError, 0, p.q[..., :64].contiguous())
    refused(ValueError, 1, p.kc.transpose(2, 3))
    refused(ValueError, 2, p.vc[:-1])
    refused(ValueError, 2, p.vc.transpose(1, 2).contiguous().transpose(1, 2))
    refused(TypeError, 3, _i32(p.table).long())
    refused(ValueError, 3, _i32(p.table)[:-1])
    refused(ValueError, 4, _i32(p.cu)[:-1])
    refused(ValueError, 5, _i32(p.lk).cpu())
    with pytest.raises(ValueError):
        p.run(out=torch.empty_like(p.q)[:, :-1])
    with pytest.raises(fa.FatAttnError):
        p.run(workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    k = _bf16(np.random.default_rng(1), 3, 2, 128)
    with pytest.raises(ValueError):
        fa.fat_paged_append(k, k, p.kc, p.vc, _i32([1, 2]))
    with pytest.raises(ValueError):
        fa.fat_paged_append(k[:, :1], k, p.kc, p.vc, _i32([1, 2, 3]))
    with pytest.raises(ValueError):
        fa.fat_rope_embed(k, _i32([1, 2]), fa.fat_rope_init(64))
    with pytest.raises(TypeError):
        fa.fat_rope_embed(k, torch.zeros(3, device=DEV), fa.fat_rope_init(64))
    with pytest.raises(TypeError):  # a rotation that fat_rope_init has not made
        fa.fat_rope_embed(k, _i32([1, 2, 3]), bytes(1040))
    with pytest.raises(TypeError):
        p.run(max_q="1")
    with pytest.raises(ValueError):
        p.run(max_k=1 << 40)
    with pytest.raises(fa.FatAttnError):
        p.run(max_q=-1)
    with pytest.raises(ValueError):
        fa.fat_paged_plan(_i32([1, 2]), _i32([1]), _i32([0]), _i32([[0], [0]]), 16, 4, 4)


# ---- together -----------------------------------------------------------------------------------
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(graph):
    """Prompts in chunks and then single tokens through plan, append and attention equals, row by
    row, causal attention with the document rotation over the whole sequences at once."""
    rng = np.random.default_rng(31)
    hq, hkv, d, page, pages = 4, 2, 64, 16, 64
    lens = [75, 40, 1, 130]
    n = len(lens)
    docs = [_bf16(rng, m, hq + 2 * hkv, d) for m in lens]
    packed = torch.cat(docs)
    cu = _i32(np.concatenate([[0], np.cumsum(lens)]))
    rope_q = fa.fat_rope_apply(packed[:, :hq].contiguous(), cu, max(lens))
    rope_k = fa.fat_rope_apply(packed[:, hq:hq + hkv].contiguous(), cu, max(lens))
    want, _ = fa.fat_xattn_fwd(rope_q, rope_k, packed[:, hq + hkv:].contiguous(), cu, cu, max(lens),
                               max(lens), causal=True, softmax_scale=d ** -0.5)
    steps = [[60, 0, 1, 0], [10, 33, 0, 64], [1, 1, 0, 64], [1, 1, 0, 1], [1, 1, 0, 1],
             [1, 1, 0, 0], [1, 1, 0, 0], [0, 1, 0, 0], [0, 1, 0, 0]]
    assert [sum(c) for c in zip(*steps)] == lens
    kc, vc = _make_cache(pages, page, hkv, d, "token", float("nan"))
    free = torch.as_tensor(rng.permutation(pages).astype(np.int32)).to(DEV)
    table = torch.full((n, 10), -1, dtype=torch.int32, device=DEV)
    rope = fa.fat_rope_init(d)
    cap = max(sum(s) for s in steps)
    qkv = torch.zeros((cap, hq + 2 * hkv, d), dtype=torch.bfloat16, device=DEV)
    ctx, new = _i32([0] * n), _i32([0] * n)
    freeb = free.clone()
    bufs = dict(cu_seqlens_q=_i32([0] * (n + 1)), seqlens_k=_i32([0] * n),
                positions=_i32([0] * cap), slots=_i32([0] * cap), counts=_i32([0, 0]))
    out = torch.zeros((cap, hq, d), dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros((hq, cap), device=DEV)
    qr = torch.zeros((cap, hq, d), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(1, fa.fat_paged_attn_workspace_size(qr, kc, bufs["cu_seqlens_q"], cap,
                                                             160)), dtype=torch.uint8, device=DEV)

    def step():
        cu_q, lk, pos, slots, _ = fa.fat_paged_plan(ctx, new, freeb, table, page, pages, cap, **bufs)
        q, k, v = qkv.split([hq, hkv, hkv], dim=1)
        fa.fat_paged_append(k, v, kc, vc, slots, q=q, positions=pos, rope=rope, q_out=qr)
        fa.fat_paged_attn(qr, kc, vc, table, cu_q, lk, cap, 160, causal=True,
                          softmax_scale=d ** -0.5, out=out, lse=lse, workspace=ws)

    g = None
    if graph:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        kc.fill_(float("nan"))
        vc.fill_(float("nan"))
        table.fill_(-1)
    done = [0] * n
    got = [[] for _ in range(n)]
    for s in steps:
        rows = [docs[i][done[i]:done[i] + s[i]] for i in range(n)]
        qkv.fill_(float("nan"))  # padding rows hold anything
        qkv[:sum(s)] = torch.cat(rows)
        ctx.copy_(_i32(done))
        new.copy_(_i32(s))
        if g is None:
            step()
        else:
            g.replay()
        assert _errors() == 0
        taken = int(bufs["counts"][0])
        freeb.copy_(torch.cat([freeb[taken:], freeb[:taken]]))
        at = 0
        for i in range(n):
            got[i].append(out[at:at + s[i]].clone())
            at += s[i]
            done[i] += s[i]
    res = torch.cat([torch.cat(x) for x in got])
    # both are within one bf16 rounding of P and of the result of the same exact values (the rotated
    # queries and keys are equal bit for bit): 4 half steps of the weights' |V| at most
    err = (res.double() - want.double()).abs()
    v = packed[:, hq + hkv:].double().abs().amax()
    assert (err <= 2.0 ** -8 * 2 * (want.double().abs() + v)).all()
    assert err.mean() < 2.0 ** -9
