"""The output layer's cross-entropy without a GPU: what is refused on the host through the C ABI, and the
fp64 reference against autograd and differences."""
import ctypes

import pytest
import torch

import attention_relative_position_gb300 as fa
from attention_relative_position_gb300 import _build
from oracle import linear_ce

FAKE = 1 << 20  # aligned non-null host value; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.load()


def _shape(**kw):
    s = dict(rows=4, vocab=100, dim=64, hidden_stride=64, weight_stride=64, logit_scale=1.0,
             z_loss=0.0)
    s.update(kw)
    return fa._LinearCeShape(*s.values(), None)


BAD_SHAPES = [dict(rows=-1), dict(vocab=0), dict(vocab=-5), dict(dim=0), dict(dim=60), dict(dim=-8),
              dict(hidden_stride=56), dict(hidden_stride=68), dict(weight_stride=0),
              dict(weight_stride=1 << 38), dict(logit_scale=0.0), dict(logit_scale=-1.0),
              dict(logit_scale=float("inf")), dict(logit_scale=float("nan")), dict(z_loss=-1.0),
              dict(z_loss=float("nan"))]
TOO_LARGE = [dict(dim=65544, hidden_stride=65544, weight_stride=65544), dict(vocab=1 << 29),
             dict(rows=1 << 29), dict(rows=1 << 28, vocab=1 << 16)]


def test_exports(lib):
    for name in ("fat_linear_cross_entropy_fwd", "fat_linear_cross_entropy_bwd",
                 "fat_linear_cross_entropy_workspace_size"):
        assert hasattr(lib, name) and hasattr(fa, name) and name in fa.__all__, name


def test_shape_refusals(lib):
    size = ctypes.c_size_t(1 << 40)
    for bad, code in [(b, -2) for b in BAD_SHAPES] + [(b, -5) for b in TOO_LARGE]:
        sh = _shape(**bad)
        assert lib.fat_linear_cross_entropy_workspace_size(sh, 0) == 0, bad
        assert lib.fat_linear_cross_entropy_workspace_size(sh, 1) == 0, bad
        assert lib.fat_linear_cross_entropy_fwd(sh, *[FAKE] * 4, size, FAKE, FAKE) == code, bad
        assert lib.fat_linear_cross_entropy_bwd(sh, *[FAKE] * 5, 1.0, FAKE, size, FAKE, FAKE) == code
    assert lib.fat_linear_cross_entropy_fwd(None, *[FAKE] * 4, size, FAKE, FAKE) == -1
    assert lib.fat_linear_cross_entropy_bwd(None, *[FAKE] * 5, 1.0, FAKE, size, FAKE, FAKE) == -1


def test_pointer_refusals(lib):
    size = ctypes.c_size_t(1 << 40)
    sh = _shape()
    for i in range(4):  # hidden, weight, target, workspace
        args = [FAKE] * 4
        args[i] = None
        assert lib.fat_linear_cross_entropy_fwd(sh, *args, size, FAKE, FAKE) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 128), (4, 2), (5, 2)):
        args = [FAKE] * 4 + [size] + [FAKE] * 2
        args[i if i < 4 else i + 1] = FAKE + off
        assert lib.fat_linear_cross_entropy_fwd(sh, *args) == -2, i
    # hidden, weight, target, lse, dloss, grad_scale, workspace, bytes, dhidden, dweight
    good = [FAKE] * 5 + [1.0, FAKE, size, FAKE, FAKE]
    for i in (0, 1, 2, 3, 6):
        args = list(good)
        args[i] = None
        assert lib.fat_linear_cross_entropy_bwd(sh, *args) == -1, i
    for i, off in ((0, 8), (1, 8), (2, 2), (3, 2), (4, 2), (6, 128), (8, 8), (9, 8)):
        args = list(good)
        args[i] = FAKE + off
        assert lib.fat_linear_cross_entropy_bwd(sh, *args) == -2, i


def test_nothing_to_do(lib):
    size = ctypes.c_size_t(0)
    assert lib.fat_linear_cross_entropy_fwd(_shape(rows=0), *[None] * 4, size, None, None) == 0
    assert lib.fat_linear_cross_entropy_bwd(_shape(rows=0), *[None] * 5, 1.0, None, size, FAKE,
                                            None) == 0
    assert lib.fat_linear_cross_entropy_bwd(_shape(), *[None] * 5, 1.0, None, size, None, None) == 0


@pytest.mark.parametrize("z_loss,scale", [(0.0, 1.0), (1e-2, 0.3)])
def test_reference(z_loss, scale):
    g = torch.Generator().manual_seed(5)
    h = torch.randn(11, 24, generator=g).double().requires_grad_()
    w = torch.randn(37, 24, generator=g).double().requires_grad_()
    t = torch.randint(0, 37, (11,), generator=g)
    t[3], t[8] = -100, 37
    dloss = torch.rand(11, generator=g).double()
    ok = (t >= 0) & (t < 37)
    z = scale * h @ w.t()
    lse = torch.logsumexp(z, 1)
    want = torch.nn.functional.cross_entropy(z[ok], t[ok], reduction="none") + z_loss * lse[ok] ** 2
    loss, got_lse = linear_ce.forward(h.detach(), w.detach(), t, z_loss, scale)
    assert torch.allclose(loss[ok], want, rtol=1e-13, atol=1e-13) and (loss[~ok] == 0).all()
    assert torch.allclose(got_lse, lse, rtol=1e-13)
    (0.25 * (want * dloss[ok]).sum()).backward()
    dh, dw, eh, ew = linear_ce.backward(h.detach(), w.detach(), t, dloss, z_loss, scale, 0.25)
    assert torch.allclose(dh, h.grad, rtol=1e-11, atol=1e-13)
    assert torch.allclose(dw, w.grad, rtol=1e-11, atol=1e-13)
    assert (eh == 0).all() and (ew == 0).all()
    # the bound of the roundings covers a gradient of logits that is off by 2^-8 everywhere
    _, _, eh, ew = linear_ce.backward(h.detach(), w.detach(), t, dloss, z_loss, scale, 0.25,
                                      rounding=2.0 ** -8)
    assert (dh.abs() * 2.0 ** -8 <= eh * (1 + 1e-12)).all()
    assert (dw.abs() * 2.0 ** -8 <= ew * (1 + 1e-12)).all()
    # differences
    u, e = torch.randn(11, 24, generator=g).double(), 1e-6
    f = lambda x: (0.25 * dloss * linear_ce.forward(x, w.detach(), t, z_loss, scale)[0]).sum()  # noqa: E731
    slope = (f(h.detach() + e * u) - f(h.detach() - e * u)) / (2 * e)
    assert abs(slope - (dh * u).sum()) < 1e-7
