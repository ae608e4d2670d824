"""Pins of the cache, attention and norm oracle (no GPU): worked groups, closed forms, brute force."""
import math

import numpy as np
import pytest

import oracle.kv4 as O


def test_bf16_rounds_to_nearest_even():
    x = np.array([1.0, 1 + 2 ** -8, 1 + 3 * 2 ** -8, 1 + 2 ** -8 + 2 ** -20, -1 - 2 ** -8], np.float32)
    assert O.bf16(x).tolist() == [1.0, 1.0, 1 + 2 ** -6, 1 + 2 ** -7, -1.0]


def test_a_ramp_is_kept_exactly():
    """Values 0, 1, .., 15: s = 1, o = 8, codes 0..15."""
    x = np.tile(np.arange(16, dtype=np.float32), 2)
    s, o, n = O.quantise(x, 32)
    assert s.tolist() == [1.0] and o.tolist() == [8.0] and n.tolist() == x.astype(int).tolist()
    assert O.stored(x, 32).tolist() == x.tolist()


def test_a_worked_group():
    """Range -3 .. 4.5 gives s = 0.5, o = 1; 0.3 -> rint(-1.4) + 8 = 7 -> 0.5; ties go to even codes."""
    x = np.zeros(32, np.float32)
    x[:6] = [-3.0, 4.5, 0.3, 0.25, 0.75, 1.25]
    s, o, n = O.quantise(x, 32)
    assert s.tolist() == [0.5] and o.tolist() == [1.0]
    assert n[:6].tolist() == [0, 15, 7, 6, 8, 8]   # (0.25 - 1) / 0.5 = -1.5 -> -2; -0.5 -> -0; 0.5 -> 0


def test_constant_tiny_and_broken_groups():
    x = np.full((3, 32), 3.0, np.float32)
    x[1] = np.linspace(0, 2 ** -130, 32)
    x[2, 5] = np.nan
    s, o, n = O.quantise(x, 32)
    assert (s == 0).all() and o[0] == 3.0 and np.isnan(o[2]) and (n == 8).all()
    assert (O.stored(x, 32)[0] == 3.0).all() and np.isnan(O.stored(x, 32)[2]).all()


@pytest.mark.parametrize("gs", [32, 64, 128])
def test_error_is_half_a_step_plus_the_offset_rounding(gs):
    x = np.random.default_rng(gs).normal(size=(200, 128)).astype(np.float32) + np.float32(0.7)
    s, o, _ = O.quantise(x, gs)
    step, off = np.repeat(s, gs, -1), np.abs(np.repeat(o, gs, -1))
    # the range's ends lie up to 7.5 relative roundings of s plus one of o outside the codes' range
    assert (np.abs(O.stored(x, gs) - x) <= step * (0.5 + 8 * 2.0 ** -8) + off * 2.0 ** -8).all()


def test_attention_by_scalar_loops():
    r = np.random.default_rng(1)
    q, K, V = r.normal(size=(3, 4, 8)), r.normal(size=(6, 2, 8)), r.normal(size=(6, 2, 8))
    out, mag, size = O.attention(q, K, V, [3, 4, 5], 0.3, window=4)
    for i, p in enumerate((3, 4, 5)):
        for h in range(4):
            ts = [t for t in range(6) if p - 4 < t <= p]
            w = [math.exp(0.3 * sum(q[i, h, d] * K[t, h // 2, d] for d in range(8))) for t in ts]
            for d in range(8):
                assert math.isclose(out[i, h, d], sum(a * V[t, h // 2, d] for a, t in zip(w, ts)) / sum(w), rel_tol=1e-12)
    assert (mag >= np.abs(out) - 1e-12).all() and (size > 0).all()


def test_attention_of_rows_that_see_nothing_one_token_and_shifted_scores():
    r = np.random.default_rng(2)
    q, K, V = r.normal(size=(2, 2, 8)), r.normal(size=(5, 1, 8)), r.normal(size=(5, 1, 8))
    out = O.attention(q, K, V, [-1, 0], 1.0)[0]
    assert (out[0] == 0).all() and np.allclose(out[1], V[0])
    # a constant added to every key moves all scores of a query together
    a, b = (O.attention(q, k, V, [4, 4], 1.0)[0] for k in (K, K + 0.5))
    assert np.allclose(a, b)


def test_norm_residual_closed_forms():
    b = np.array([[3.0, 4.0, 0.0, 0.0]])
    h, x = O.norm_residual(b, None, None, 2.0, np.ones(4), np.array([1.0, 1, 1, 2]), 0.0)
    assert np.allclose(h, 2 * b / 2.5) and np.allclose(x, b / 2.5 * [1, 1, 1, 2])
    h, x = O.norm_residual(b, b, np.zeros((1, 4)), 0.5, None, None, 0.0, gate_sigmoid=True)
    assert np.allclose(h, 1.25 * b) and x is None
    h, x = O.norm_residual(None, b, None, 1.0, None, np.ones(4), 0.0)
    assert (h == b).all() and np.allclose((x * x).mean(), 1)
