"""Pins of the serving oracle: closed forms and limits that it must meet by itself (CPU)."""
import numpy as np
import pytest

from oracle import muse_oracle as mo
from oracle import serving_oracle as so

SECTIONS = [(64,), (16, 24, 24), (10, 5), (1, 2, 3, 4)]


@pytest.mark.parametrize("sections", SECTIONS)
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("ladder", [False, True])
def test_rope_is_a_rotation_and_its_inverse_undoes_it(sections, adjacent, ladder):
    rng = np.random.default_rng(1)
    X = rng.standard_normal((2, 3, 5, 128))
    pos = rng.integers(-(1 << 31), 1 << 31, (2, len(sections), 5))
    kw = dict(adjacent=adjacent, axis_ladder=ladder)
    Y = so.rope(X, pos, sections, 1e4, **kw)
    np.testing.assert_allclose((Y ** 2).sum(-1), (X ** 2).sum(-1), rtol=1e-13)
    np.testing.assert_allclose(so.rope(Y, pos, sections, 1e4, inverse=True, **kw), X, atol=1e-14)
    P = sum(sections)
    assert np.array_equal(Y[..., 2 * P:], X[..., 2 * P:])


def test_rope_products_depend_on_differences_of_positions():
    """One axis: q.k after turning depends on the two positions' difference only."""
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 1, 64))
    at = lambda x, p: so.rope(x, np.array([[[p]]]), (32,), 1e4)
    near = (at(q, 7) * at(k, 3)).sum()
    far = (at(q, 2_000_000_007) * at(k, 2_000_000_003)).sum()
    np.testing.assert_allclose(far, near, atol=1e-12)


def test_rope_gradient_against_differences():
    rng = np.random.default_rng(3)
    X, W = rng.standard_normal((2, 1, 2, 3, 64))
    pos = rng.integers(0, 100, (1, 2, 3))
    f = lambda x: (so.rope(x, pos, (10, 20), 100.0) * W).sum()
    G = so.rope(W, pos, (10, 20), 100.0, inverse=True)
    for idx in [(0, 0, 0, 0), (0, 1, 2, 31), (0, 1, 1, 63), (0, 0, 2, 40)]:
        d = np.zeros_like(X)
        d[idx] = 1e-4
        np.testing.assert_allclose((f(X + d) - f(X - d)) / 2e-4, G[idx], atol=1e-9)


def test_quantised_values_are_within_half_a_step_and_fixed_points():
    rng = np.random.default_rng(4)
    X = so.bf16(rng.standard_normal((50, 128)) * np.exp(4 * rng.standard_normal((50, 1))))
    q, step = so.quantise(X)
    Y = so.held(X)
    # the largest of a group may be cut by the step's rounding (2^-9 of 7 steps, below half a one)
    assert (np.abs(Y - X) <= 0.5 * np.repeat(step, 32, -1) * (1 + 1e-12)).all()
    assert np.abs(q).max() == 7 and (np.abs(q).reshape(50, 4, 32).max(-1) == 7).all()


def test_quantise_edges():
    x = np.zeros((1, 64))
    assert (so.held(x) == 0).all()
    x[0, 3], x[0, 40] = np.inf, 7.0
    x[0, 41:44] = 0.5, 1.5, -2.5          # ties go to the even code
    y = so.held(x)
    assert np.isnan(y[0, :32]).all()
    assert y[0, 40:44].tolist() == [7.0, 0.0, 2.0, -2.0]


@pytest.mark.parametrize("D,Dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_tile_layout_places_every_value_once(D, Dv):
    (kb, ks, kst), (vb, vs, vst) = so.tile_layout(D, Dv)
    codes = np.concatenate([(2 * kb + ks // 4).ravel(), (2 * vb + vs // 4).ravel()])
    assert np.array_equal(np.sort(codes), np.arange(2 * 16 * (D + Dv)))
    steps = np.concatenate([np.unique(kst), np.unique(vst)])
    assert np.array_equal(np.sort(steps), np.arange(16 * (D + Dv), 18 * (D + Dv), 2))


def test_attend_over_exact_values_is_causal_softmax_attention():
    """The newest N = T rows over a cache of T tokens is plain causal attention."""
    rng = np.random.default_rng(5)
    T, D = 12, 8
    Q, K, V = rng.standard_normal((3, 1, 2, T, D))
    O, lse, _, _ = so.cache_attend(Q, [K[0]], [V[0]], [T], [T], 0.3)
    for h in range(2):
        np.testing.assert_allclose(O[0, h], mo.exact_attention(Q[0, h], K[0, h], V[0, h], 0.3,
                                                               causal=True), atol=1e-12)
        x = 0.3 * Q[0, h] @ K[0, h].T
        x[np.triu_indices(T, 1)] = -np.inf
        np.testing.assert_allclose(lse[0, h], np.log(np.exp(x).sum(-1)), atol=1e-12)
