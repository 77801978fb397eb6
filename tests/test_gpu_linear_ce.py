"""GPU parity of the output layer's cross-entropy (loss without logits, its gradient) against fp64."""
import math

import numpy as np
import pytest
import torch

import attention_relative_position_gb300 as fa
from oracle import linear_ce

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _clean_error_word():
    torch.cuda.synchronize()
    fa.fat_attn_get_device_error()


def _errors():
    torch.cuda.synchronize()
    return fa.fat_attn_get_device_error()


def _inputs(rows, vocab, dim, seed=0, ignored=0.0, std=2.0):
    g = torch.Generator(device=DEV).manual_seed(1000 * rows + 10 * vocab + dim + seed)
    h = torch.randn(rows, dim, generator=g, device=DEV).to(torch.bfloat16)
    w = (std * dim ** -0.5 * torch.randn(vocab, dim, generator=g, device=DEV)).to(torch.bfloat16)
    t = torch.randint(0, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    drop = torch.rand(rows, generator=g, device=DEV) < ignored
    return h, w, torch.where(drop, -100, t).to(torch.int32)


# A logit is a sum of dim exact products in fp32: dim / 16 steps of 16 products, each rounded or cut
# to 2^-23 of what was summed so far, and 16 more for the order within a step, all relative to
# A = scale * sum |h w|. Everything else of lse: the scaled logit (2^-24 of it, twice), exponentials
# (2^-22, hardware), their sums over up to 256 values a tile and the merge over the tiles (a rounding
# of 2^-24 for each term of a thread's sum: fewer than 512 in all), logarithm and last product (a few).
def _logit_tol(h, w, scale):
    most = max(float((h[r:r + 2048].float().abs() @ w.float().abs().t()).max())
               for r in range(0, h.shape[0], 2048))
    return (h.shape[1] / 16 + 16) * 2.0 ** -23 * scale * most


def _check_fwd(h, w, t, z_loss=0.0, scale=1.0, bits=0, **kw):
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t, z_loss=z_loss, logit_scale=scale, **kw)
    assert _errors() == bits
    want, want_lse = linear_ce.forward(h, w, t, z_loss, scale)
    tz = _logit_tol(h, w, scale)
    tol = tz + 2.0 ** -24 * (4 * 1.45 * float(want_lse.abs().max()) + 4 * 1.45 * tz + 600)
    assert (lse.double() - want_lse).abs().max() <= tol
    # loss: the target's logit too, and z_loss lse^2 (three roundings)
    tol = 2 * tol + z_loss * (2 * want_lse.abs().max() + tol) * tol + 4 * 2.0 ** -24 * want.abs().max()
    assert (loss.double() - want).abs().max() <= tol
    assert (loss[t < 0] == 0).all()
    return loss, lse


SHAPES = [(1, 1, 8), (1, 300, 64), (2, 16, 16), (3, 17, 72), (37, 5000, 768), (255, 257, 64),
          (256, 256, 128), (257, 513, 136), (300, 2000, 520), (5, 40001, 64), (1, 131072, 64),
          (129, 20000, 1032), (700, 1025, 2048), (2500, 3001, 192), (8, 127, 64), (9, 128, 64), (16, 129, 64),
          (17, 511, 64), (64, 513, 1032), (128, 3000, 264), (1537, 700, 200), (2000, 300, 24)]


@pytest.mark.parametrize("rows,vocab,dim", SHAPES)
def test_forward(rows, vocab, dim):
    h, w, t = _inputs(rows, vocab, dim, ignored=0.2 if rows > 2 else 0.0)
    _check_fwd(h, w, t, z_loss=1e-4 if rows % 2 else 0.0, scale=0.5 if dim == 64 else 1.0)


def _check_bwd(h, w, t, dloss=None, z_loss=0.0, scale=1.0, grad_scale=1.0, bits=0, **kw):
    clean = torch.where(((t >= 0) & (t < w.shape[0]))[:, None], h, 0)
    _, lse = linear_ce.forward(clean, w, t, z_loss, scale)
    lse = lse.float()
    dh, dw = fa.fat_linear_cross_entropy_bwd(h, w, t, lse, dloss=dloss, z_loss=z_loss,
                                             logit_scale=scale, grad_scale=grad_scale, **kw)
    assert _errors() == bits
    # The softmax: logits as above, what the exponent takes on the way (the scaled logit and lse, 2^-24
    # each, rounded and subtracted, in log2 units), the exponential and two products (2^-22). dz is
    # rounded to bf16 (2^-8 of it).
    big = float(lse.abs().max()) + _logit_tol(clean, w, scale)
    rel = _logit_tol(clean, w, scale) + 2.0 ** -24 * (4 * 1.45 * big + 8)
    xh, xw, eh, ew = linear_ce.backward(h, w, t, dloss, z_loss, scale, grad_scale, lse=lse, rel=rel,
                                        rounding=2.0 ** -8)
    # sums in fp32 (each of the products' steps as above, relative to the sum of magnitudes, which
    # is at most 2^8 times the bound of the roundings), and the result's own rounding
    for got, want, off, n in ((dh, xh, eh, w.shape[0]), (dw, xw, ew, h.shape[0])):
        if got is None:
            continue
        tol = off * (1 + 256 * (n / 16 + 32) * 2.0 ** -23) * 1.01 + 2.0 ** -8 * want.abs() + 1e-37
        bad = (got.double() - want).abs() > tol
        assert not bad.any(), (int(bad.sum()), float(((got.double() - want).abs() / tol).max()))
    return dh, dw


@pytest.mark.parametrize("rows,vocab,dim", SHAPES)
def test_backward(rows, vocab, dim):
    h, w, t = _inputs(rows, vocab, dim, seed=1, ignored=0.2 if rows > 2 else 0.0)
    dloss = torch.rand(rows, device=DEV) - 0.3 if rows % 3 else None
    _check_bwd(h, w, t, dloss, z_loss=1e-3 if rows % 2 else 0.0, scale=0.5 if dim == 64 else 1.0,
               grad_scale=1.0 / rows)


# several pieces of the vocabulary, several blocks of rows
@pytest.mark.parametrize("rows,vocab,dim", [(16384, 9001, 64), (16700, 9001, 72), (33000, 520, 136),
                                            (3000, 60000, 40)])
def test_pieces(rows, vocab, dim):
    h, w, t = _inputs(rows, vocab, dim, ignored=0.1)
    _check_fwd(h, w, t, z_loss=1e-4)
    _check_bwd(h, w, t, z_loss=1e-4, grad_scale=1.0 / rows)


def test_odd_rows_with_other_strides():
    """Many rows of an odd number of 16 bytes: rows a stride apart that needs no copy, and one that does."""
    for pad in (8, 16):
        h = torch.randn(1600, 72 + pad, device=DEV).to(torch.bfloat16)[:, :72]
        w = (0.2 * torch.randn(500, 72 + pad, device=DEV)).to(torch.bfloat16)[:, :72]
        t = torch.randint(0, 500, (1600,), device=DEV).to(torch.int32)
        _check_fwd(h, w, t)
        _check_bwd(h, w, t)
    # an even number of them, rows an odd number apart
    h = torch.randn(1600, 72, device=DEV).to(torch.bfloat16)[:, :64]
    w = (0.2 * torch.randn(500, 72, device=DEV)).to(torch.bfloat16)[:, :64]
    _check_fwd(h, w, t)
    _check_bwd(h, w, t)


def test_strided_rows():
    wide_h = torch.randn(100, 3, 96, device=DEV).to(torch.bfloat16)
    wide_w = torch.randn(777, 104, device=DEV).to(torch.bfloat16) * 0.2
    h, w = wide_h[:, 1, :72], wide_w[:, 8:80]
    t = torch.randint(0, 777, (100,), device=DEV).to(torch.int32)
    _check_fwd(h, w, t)
    _check_bwd(h, w, t)


def test_one_gradient_at_a_time():
    h, w, t = _inputs(300, 700, 136)
    lse = fa.fat_linear_cross_entropy_fwd(h, w, t)[1]
    dh, dw = fa.fat_linear_cross_entropy_bwd(h, w, t, lse)
    a, none = fa.fat_linear_cross_entropy_bwd(h, w, t, lse, want_dweight=False)
    assert none is None and torch.equal(a, dh)
    none, b = fa.fat_linear_cross_entropy_bwd(h, w, t, lse, want_dhidden=False)
    assert none is None and torch.equal(b, dw)
    assert fa.fat_linear_cross_entropy_bwd(h, w, t, lse, want_dhidden=False,
                                           want_dweight=False) == (None, None)


def test_ignored_rows_may_hold_anything():
    h, w, t = _inputs(500, 900, 200, ignored=0.4)
    drop = t < 0
    bad = h.clone()
    bad[drop] = float("nan")
    bad[torch.nonzero(drop)[0]] = float("inf")
    loss, _ = fa.fat_linear_cross_entropy_fwd(bad, w, t)
    assert torch.isfinite(loss).all() and (loss[drop] == 0).all()
    lse = fa.fat_linear_cross_entropy_fwd(h, w, t)[1]
    want = fa.fat_linear_cross_entropy_bwd(h, w, t, lse)
    lse_bad = torch.where(drop, float("nan"), lse)
    got = fa.fat_linear_cross_entropy_bwd(bad, w, t, lse_bad)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0][drop] == 0).all()
    # no row counts
    none = torch.full_like(t, -1)
    dh, dw = fa.fat_linear_cross_entropy_bwd(bad, w, none, lse_bad)
    assert (dh == 0).all() and (dw == 0).all()


def test_nan_shows():
    h, w, t = _inputs(300, 500, 64)
    h[7, 3] = float("nan")
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    assert torch.isnan(loss[7]) and torch.isnan(lse[7])
    assert torch.isfinite(loss[:7]).all() and torch.isfinite(loss[8:]).all()


def test_targets_beyond_the_vocabulary():
    h, w, t = _inputs(64, 300, 64)
    t[5], t[9] = 300, 2 ** 31 - 1
    loss, lse = _check_fwd(h, w, t, bits=fa.FAT_DEVERR_INDEX)
    assert loss[5] == 0 and loss[9] == 0
    dh, _ = _check_bwd(h, w, t, bits=fa.FAT_DEVERR_INDEX)
    assert (dh[5] == 0).all() and (dh[9] == 0).all()


def test_no_rows():
    h, w, t = _inputs(4, 40, 64)
    e = h[:0]
    loss, lse = fa.fat_linear_cross_entropy_fwd(e, w, t[:0])
    assert loss.numel() == 0 and lse.numel() == 0
    dw = torch.full_like(w, 7.0)
    dh, dw = fa.fat_linear_cross_entropy_bwd(e, w, t[:0], lse, dweight=dw)
    assert dh.shape == e.shape and (dw == 0).all() and _errors() == 0


def test_large_logits():
    # logits of hundreds and of 1e5: the softmax is one entry's, the loss exact to the logits' rounding
    for std in (200.0, 5e4):
        h, w, t = _inputs(200, 3000, 64, std=std)
        _check_fwd(h, w, t)


def test_against_the_loss_of_logits():
    # the same numbers as the library's loss over logits, up to those logits' rounding to bf16
    h, w, t = _inputs(400, 1024, 256, ignored=0.1)
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t, z_loss=1e-3)
    z = (h.float() @ w.float().t()).to(torch.bfloat16)
    want, want_lse, _ = fa.fat_cross_entropy(z, t, z_loss=1e-3)
    off = 2.0 ** -8 * float(z.float().abs().max())
    assert (lse - want_lse).abs().max() <= off
    assert (loss - want).abs().max() <= 2.1 * off


def test_gradient_against_differences():
    h, w, t = _inputs(40, 300, 64, ignored=0.2)
    lse = fa.fat_linear_cross_entropy_fwd(h, w, t, z_loss=1e-2)[1]
    dh, dw = fa.fat_linear_cross_entropy_bwd(h, w, t, lse, z_loss=1e-2)
    g = torch.Generator(device=DEV).manual_seed(3)
    for grad, x in ((dh, h), (dw, w)):
        u = torch.randn(x.shape, generator=g, device=DEV).double()
        e = 1e-4
        args = [(x.double() + s * e * u, w if x is h else h) for s in (1, -1)]
        total = [linear_ce.forward(*(a if x is h else a[::-1]), t, 1e-2)[0].sum() for a in args]
        slope = (total[0] - total[1]) / (2 * e)
        # each entry off by 2^-8 of it twice (dz and the result), and less than that in all
        assert abs(slope - (grad.double() * u).sum()) <= 2 ** -7 * (grad.double() * u).abs().sum()


def test_repeatable_and_captured():
    h, w, t = _inputs(600, 5000, 264, ignored=0.1)
    first = fa.fat_linear_cross_entropy_fwd(h, w, t)
    grads = fa.fat_linear_cross_entropy_bwd(h, w, t, first[1])
    for _ in range(3):
        assert torch.equal(fa.fat_linear_cross_entropy_fwd(h, w, t)[0], first[0])
        again = fa.fat_linear_cross_entropy_bwd(h, w, t, first[1])
        assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])
    out = [torch.empty_like(x) for x in (*first, *grads)]
    ws = [torch.empty(fa.fat_linear_cross_entropy_workspace_size(600, 5000, 264, backward=b),
                      dtype=torch.uint8, device=DEV) for b in (False, True)]
    hs, ts = torch.zeros_like(h), torch.zeros_like(t)

    def step():
        fa.fat_linear_cross_entropy_fwd(hs, w, ts, loss=out[0], lse=out[1], workspace=ws[0])
        fa.fat_linear_cross_entropy_bwd(hs, w, ts, out[1], dhidden=out[2], dweight=out[3],
                                        workspace=ws[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hs.copy_(h)
    ts.copy_(t)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(out, (*first, *grads)):
        assert torch.equal(got, want)


def test_on_a_given_stream():
    h, w, t = _inputs(100, 900, 128)
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    dh, dw = fa.fat_linear_cross_entropy_bwd(h, w, t, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        l2, e2 = fa.fat_linear_cross_entropy_fwd(h, w, t, stream=s)
        g2 = fa.fat_linear_cross_entropy_bwd(h, w, t, e2, stream=s)
    s.synchronize()
    assert torch.equal(l2, loss) and torch.equal(g2[0], dh) and torch.equal(g2[1], dw)


@pytest.mark.parametrize("rows,vocab,dim", [(1, 3000, 64), (128, 500, 72), (300, 700, 136), (1600, 520, 72),
                                            (17000, 5000, 40)])
def test_workspace_of_the_given_size(rows, vocab, dim):
    """Nothing is written behind the bytes that the size names, and what they held does not matter."""
    h, w, t = _inputs(rows, vocab, dim, ignored=0.1)
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    want = (loss, lse, *fa.fat_linear_cross_entropy_bwd(h, w, t, lse))
    for fill in (0xff, 0x7f):
        ws = [torch.full((fa.fat_linear_cross_entropy_workspace_size(rows, vocab, dim, backward=b) + 4096,),
                         fill, dtype=torch.uint8, device=DEV) for b in (False, True)]
        got = (*fa.fat_linear_cross_entropy_fwd(h, w, t, workspace=ws[0][:-4096]),
               *fa.fat_linear_cross_entropy_bwd(h, w, t, lse, workspace=ws[1][:-4096]))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert all((x[-4096:] == fill).all() for x in ws) and _errors() == 0
        for b in (False, True):  # a byte less is refused
            with pytest.raises(fa.FatAttnError):
                if b:
                    fa.fat_linear_cross_entropy_bwd(h, w, t, lse, workspace=ws[1][:-4097])
                else:
                    fa.fat_linear_cross_entropy_fwd(h, w, t, workspace=ws[0][:-4097])


@pytest.mark.parametrize("rows", [3, 300])
def test_watchdog(rows):
    """No copies are issued: the waits run out, the status says so, and the next call is right."""
    h, w, t = _inputs(rows, 900, 128)
    _, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    try:
        fa.fat_attn_debug_set_watchdog(50_000_000, 1)
        fa.fat_linear_cross_entropy_fwd(h, w, t)
        assert _errors() == fa.FAT_DEVERR_TIMEOUT_FWD
        fa.fat_linear_cross_entropy_bwd(h, w, t, lse)
        assert _errors() == fa.FAT_DEVERR_TIMEOUT_BWD
    finally:
        fa.fat_attn_debug_set_watchdog(0, 0)
    _check_fwd(h, w, t)
    _check_bwd(h, w, t)


def test_two_calls_at_once():
    sets = [_inputs(700, 4000, 264, seed=s) for s in (1, 2)]
    want = []
    for h, w, t in sets:
        loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
        want.append((loss, lse, *fa.fat_linear_cross_entropy_bwd(h, w, t, lse)))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(8):
        got = []
        for (h, w, t), s in zip(sets, streams):
            loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t, stream=s)
            got.append((loss, lse, *fa.fat_linear_cross_entropy_bwd(h, w, t, lse, stream=s)))
        torch.cuda.synchronize()
        for g, x in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, x))


def test_arguments_are_checked():
    h, w, t = _inputs(20, 300, 64)
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    f, b = fa.fat_linear_cross_entropy_fwd, fa.fat_linear_cross_entropy_bwd
    for call, err in (
            (lambda: f(h.float(), w, t), TypeError), (lambda: f(h, w.float(), t), TypeError),
            (lambda: f(h, w, t.long()), TypeError), (lambda: f(h, w, t[:-1]), ValueError),
            (lambda: f(h, w[:, :56], t), ValueError), (lambda: f(h.cpu(), w, t), ValueError),
            (lambda: f(h[0], w, t), ValueError), (lambda: f(h[:, ::2], w[:, ::2], t), ValueError),
            (lambda: f(h, w, t, loss=loss[:-1]), ValueError), (lambda: f(h, w, t, lse=loss.double()), TypeError),
            (lambda: f(h[:, :60], w[:, :60], t), fa.FatAttnError),
            (lambda: f(h, w, t, logit_scale=0.0), fa.FatAttnError),
            (lambda: f(h, w, t, z_loss=-1.0), fa.FatAttnError),
            (lambda: f(h, w, t, loss=loss, lse=loss), fa.FatAttnError),
            (lambda: f(h, w, t, lse=h.view(torch.float32).view(-1)[:20]), fa.FatAttnError),
            (lambda: f(h, w, t, workspace=w.view(torch.uint8).view(-1)), fa.FatAttnError),
            (lambda: b(h, w, t, lse.double()), TypeError), (lambda: b(h, w, t, lse[:-1]), ValueError),
            (lambda: b(h, w, t, lse, dloss=lse[:-1]), ValueError),
            (lambda: b(h, w, t, lse, dhidden=h), fa.FatAttnError),
            (lambda: b(h, w, t, lse, dweight=w), fa.FatAttnError),
            (lambda: b(h, w, t, lse, dweight=w.float()), TypeError),
            (lambda: b(h, w, t, lse, dhidden=torch.empty_like(h)[:, :32]), ValueError),
            (lambda: b(h, w, t, lse, want_dhidden=False, dhidden=torch.empty_like(h)), ValueError)):
        with pytest.raises(err):
            call()
    assert _errors() == 0


def test_large_vocabulary_times_channels():
    """Weights and their gradient beyond 2^31 elements."""
    rows, vocab, dim = 130, 1100000, 2048
    g = torch.Generator(device=DEV).manual_seed(4)
    h = torch.randn(rows, dim, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.empty(vocab, dim, dtype=torch.bfloat16, device=DEV)
    for i in range(0, vocab, 100000):
        w[i:i + 100000] = 0.04 * torch.randn(100000, dim, generator=g, device=DEV)
    t = torch.randint(vocab - 1000, vocab, (rows,), generator=g, device=DEV).to(torch.int32)
    loss, lse = fa.fat_linear_cross_entropy_fwd(h, w, t)
    few = fa.fat_linear_cross_entropy_fwd(h[:5], w, t[:5])
    parts = [torch.logsumexp(h.double() @ w[i:i + 100000].double().t(), 1) for i in range(0, vocab, 100000)]
    want = torch.logsumexp(torch.stack(parts), 0)
    tol = 2 * _logit_tol(h, w[:2000], 1.0) + 2.0 ** -24 * 4000
    assert (lse.double() - want).abs().max() <= tol and (few[1].double() - want[:5]).abs().max() <= tol
    zt = (h.double() * w[t.long()].double()).sum(1)
    assert (loss.double() - (want - zt)).abs().max() <= 2 * tol
    dh, dw = fa.fat_linear_cross_entropy_bwd(h, w, t, lse)
    assert _errors() == 0
    # rows of the weights' gradient near both ends: each a sum over 130 rows, dz and the result rounded
    for at in (slice(0, 50), slice(vocab - 1000, vocab)):
        z = torch.exp(h.double() @ w[at].double().t() - want[:, None])
        hot = torch.arange(vocab, device=DEV)[at][None] == t[:, None]
        dz = z - hot.double()
        x = dz.t() @ h.double()
        off = (2.0 ** -8 + 1e-3) * (z + hot).t() @ h.double().abs() + 2.0 ** -8 * x.abs()
        assert ((dw[at].double() - x).abs() <= off).all()
