"""Pins of the paged-cache oracle: hand-computed maps, closed forms of the rotation, and attention
over pages against the packed cross-attention oracle's own problem."""
import numpy as np
import pytest

import oracle
from oracle import paged


def test_plan_by_hand():
    # pages of 4: request 0 has 3 of 4 slots of its page used and brings 3 tokens (one new page);
    # request 1 is new with 5 tokens (two pages); request 2 brings nothing; request 3 fills its page
    table = np.array([[9, -1, -1], [-1, -1, -1], [7, -1, -1], [5, -1, -1]])
    t, cu, lk, pos, slots, counts = paged.plan([3, 0, 2, 3], [3, 5, 0, 1], [20, 21, 22, 23], table,
                                               4, 30, 11)
    assert t.tolist() == [[9, 20, -1], [21, 22, -1], [7, -1, -1], [5, -1, -1]]
    assert cu.tolist() == [0, 3, 8, 8, 9] and lk.tolist() == [6, 5, 2, 4]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 3, 0, 0]
    assert slots.tolist() == [39, 80, 81, 84, 85, 86, 87, 88, 23, -1, -1]
    assert counts.tolist() == [3, 9]


def test_plan_without_enough_pages():
    t, cu, lk, pos, slots, counts = paged.plan([0, 0], [5, 4], [3], np.full((2, 2), -1), 4, 8, 9)
    assert t.tolist() == [[3, -1], [-1, -1]]
    assert slots.tolist() == [12, 13, 14, 15, -1, -1, -1, -1, -1] and counts.tolist() == [3, 9]


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_matches_complex_turn_and_norm(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(7, 2, 48))
    pos = np.array([0, 1, 5, 1000, 131071, 7, 7])
    y = paged.rope(x, pos, 32, interleaved=interleaved)
    first = np.arange(0, 32, 2) if interleaved else np.arange(16)
    second = first + (1 if interleaved else 16)
    z = (x[..., first] + 1j * x[..., second]) * np.exp(1j * paged.rope_angles(pos, 32))[:, None]
    np.testing.assert_allclose(y[..., first], z.real, atol=1e-12)
    np.testing.assert_allclose(y[..., second], z.imag, atol=1e-12)
    np.testing.assert_array_equal(y[..., 32:], x[..., 32:])
    np.testing.assert_array_equal(y[0], x[0])
    back = paged.rope(y, pos, 32, interleaved=interleaved, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-12)
    if interleaved:  # equal to the existing rotary oracle where both apply
        np.testing.assert_allclose(paged.rope(x, pos, 48), oracle.rope_rotate_at(x, pos, 10000.0),
                                   atol=1e-9)


def test_rope_ramp_keeps_fast_and_divides_slow_frequencies():
    a = paged.rope_angles([1.0], 64, base=10000.0, factor=8.0, ramp=(1.0, 4.0, 4096.0))[0]
    plain = paged.rope_angles([1.0], 64, base=10000.0)[0]
    turns = 4096 * plain / (2 * np.pi)
    np.testing.assert_allclose(a[turns >= 4], plain[turns >= 4], rtol=1e-14)
    np.testing.assert_allclose(a[turns <= 1], plain[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((a < plain) & (a > plain / 8))[mid].all()


def test_rope_transpose_is_the_gradient():
    """<rope(x), g> = <x, transpose(g)>, and against central differences."""
    rng = np.random.default_rng(2)
    x, g = rng.normal(size=(3, 1, 32)), rng.normal(size=(3, 1, 32))
    kw = dict(positions=np.array([3, 50, 9]), rotary_dim=16, interleaved=False, amplitude=1.2)
    grad = paged.rope(g, inverse=True, **kw)
    # channels that are only copied have gradient g; the amplitude scales the turned ones
    assert abs((paged.rope(x, **kw) * g).sum() - (x * grad).sum()) < 1e-12
    for c in (0, 7, 12, 20):
        h = np.zeros_like(x)
        h[1, 0, c] = 1e-6
        diff = ((paged.rope(x + h, **kw) - paged.rope(x - h, **kw)) * g).sum() / 2e-6
        assert abs(diff - grad[1, 0, c]) < 1e-8


def test_attention_gathers_pages_in_table_order():
    rng = np.random.default_rng(3)
    k, v = rng.normal(size=(2, 6, 4, 2, 64))
    table = np.array([[4, 1, -1], [2, 77, 0]])
    lk = np.array([6, 9])
    q = rng.normal(size=(5, 4, 64))
    cu = np.array([0, 2, 4])
    out, lse, a, s, b = paged.attention(q, k, v, table, cu, lk, causal=True, scale=0.125)
    kk = np.concatenate([k[4], k[1][:2], k[2], np.zeros((4, 2, 64)), k[0][:1]])
    vv = np.concatenate([v[4], v[1][:2], v[2], np.zeros((4, 2, 64)), v[0][:1]])
    ref, rl = oracle.xattn_fwd(oracle.XProblem(q[:4], kk, vv, cu, np.array([0, 6, 15]),
                                               causal=True, scale=0.125))
    np.testing.assert_array_equal(out, ref)
    np.testing.assert_array_equal(lse, rl)
    # one row by hand
    x = 0.125 * kk[:6, 1] @ q[1, 3]
    p = np.exp(x - x.max())
    np.testing.assert_allclose(out[1, 3], p @ vv[:6, 1] / p.sum(), atol=1e-12)
    assert (a >= np.abs(out) - 1e-12).all() and s >= np.abs(x).max() and b == 0.0
