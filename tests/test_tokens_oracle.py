"""Pins of the oracle for rotary positions, 16-bit products and log probabilities; the host part of the rotary step."""
import math
from decimal import Decimal, getcontext
from fractions import Fraction

import numpy as np
import pytest

import oracle.tokens as O
from int4_grouped_expert_router_gb300 import binding as B

PI = Fraction(Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899"))


def table(*args, **kw):
    return [int(v) % 2 ** 64 for v in B.coli_rotary_freqs(*args, device="cpu", **kw)]


def test_a_quarter_turn_a_position():
    x = np.array([[[1.0, 2.0, 7.0]]])
    quarter = [2 ** 62]
    for p, want in ((0, [1, 2]), (1, [-2, 1]), (2, [-1, -2]), (3, [2, -1]), (-1, [2, -1]), (4 * 10 ** 9 + 1, [-2, 1])):
        got = O.rotary(x, quarter, [p])[0, 0]
        assert np.allclose(got, want + [7.0], atol=1e-15), p
    assert np.allclose(O.rotary(x, quarter, [1], scale=3.0)[0, 0], [-6, 3, 7])


def test_layouts_hold_the_same_pairs():
    r = np.random.default_rng(1)
    x = r.normal(size=(3, 2, 10))
    turns = [int(v) for v in r.integers(0, 2 ** 62, size=4)]
    order = [0, 4, 1, 5, 2, 6, 3, 7, 8, 9]
    a = O.rotary(x, turns, [5, 0, 77])
    b = O.rotary(x[:, :, order], turns, [5, 0, 77], interleaved=True)
    assert np.allclose(a[:, :, order], b, atol=1e-12)
    assert np.allclose((a[:, :, :8] ** 2).sum(-1), (x[:, :, :8] ** 2).sum(-1))


def test_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(2)
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    turns = table(8, 100.0)
    dots = [float((O.rotary(q, turns, [p + 9]) * O.rotary(k, turns, [p])).sum()) for p in (0, 1, 1000, 2 ** 30)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_plan_positions():
    assert O.plan_positions(3, [5, 1, 9]) == [4, 0, 8]
    assert O.plan_positions(7, [5, 2, 1], [0, 2, 2, 5]) == [3, 4, -2, -1, 0, None, None]


SCALED = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0), "parts": dict(factor=8.0, original_len=8192, low=1.0, high=4.0)}


@pytest.mark.parametrize("scaling", list(SCALED))
@pytest.mark.parametrize("rot,base", [(2, 10000.0), (36, 500000.0), (64, 1e6), (128, 10000.0), (1024, 10.0)])
def test_the_table_of_frequencies(rot, base, scaling):
    """Against the oracle's frequencies as fractions of a turn: powers agree to a few units of 2^-53 relative, the ramp and its
    products to as many, and the fraction itself to 2 units of 2^-64."""
    getcontext().prec = 50
    got = table(rot, base, scaling=scaling, **SCALED[scaling])
    want = O.frequencies(rot, base, scaling, **SCALED[scaling])
    assert len(got) == rot // 2
    for g, f in zip(got, want):
        exact = Fraction(float(f)) / (2 * PI) * 2 ** 64
        assert abs(g - exact) <= exact * 32 / 2 ** 53 + 2


def test_parts_keep_fast_pairs_and_stretch_slow_ones():
    plain, parts = table(128, 10000.0), table(128, 10000.0, scaling="parts", factor=8.0, original_len=8192, low=1.0, high=4.0)
    turns = [8192 * t / 2 ** 64 for t in plain]
    for p, s, r in zip(plain, parts, turns):
        assert s == p if r > 4 else abs(s - p / 8) <= p / 2 ** 40 if r < 1 else p / 8 <= s <= p


@pytest.mark.parametrize("args,kw", [((3,), {}), ((0,), {}), ((1026,), {}), ((64, 1.0), {}), ((64, math.inf), {}), ((64, math.nan), {}),
                                     ((64,), dict(scaling="linear", factor=0.5)), ((64,), dict(scaling="linear", factor=math.nan)),
                                     ((64,), dict(scaling="base", factor=math.inf)), ((64, 1e300), dict(scaling="base", factor=1e300)),
                                     ((64,), dict(scaling="parts", factor=8.0)),
                                     ((64,), dict(scaling="parts", factor=8.0, original_len=10, low=4.0, high=4.0)),
                                     ((64,), dict(scaling="parts", factor=8.0, original_len=10, low=-1.0, high=4.0)),
                                     ((64,), dict(scaling="parts", factor=8.0, original_len=10, low=math.nan, high=4.0))])
def test_tables_that_are_refused(args, kw):
    with pytest.raises(B.ColiError) as e:
        B.coli_rotary_freqs(*args, device="cpu", **kw)
    assert e.value.code == B.COLI_E_INVAL


def test_an_unknown_scaling_is_refused():
    with pytest.raises(ValueError):
        B.coli_rotary_freqs(64, scaling="yes", device="cpu")


def test_activations():
    z = np.array([-50.0, -1.0, 0.0, 1.0, 50.0])
    assert np.allclose(O.act(z, "silu"), [-50 / (1 + math.exp(50)), -1 / (1 + math.e), 0, 1 / (1 + 1 / math.e), 50])
    assert np.allclose(O.act(z, "gelu"), [0, -0.15865525393145707, 0, 0.8413447460685429, 50])
    assert np.allclose(O.act(z, "gelu_tanh"), [0, -0.15880800939172324, 0, 0.8411919906082768, 50])
    assert np.array_equal(O.act(z, "relu"), [0, 0, 0, 1, 50]) and np.array_equal(O.act(z, "relu2"), [0, 0, 0, 1, 2500])


def test_linear_by_hand():
    y, z, size = O.linear([[1, 2], [0, -1]], [[3, 4], [-5, 6], [0, 1]], [10, 0, 0], "relu", [[1, 2, 3]] * 2, [[0.5, 0, 0]] * 2)
    assert np.array_equal(z, [[21, 7, 2], [6, -6, -1]]) and np.array_equal(size, [[21, 17, 2], [14, 6, 1]])
    assert np.array_equal(y, [[21.5, 14, 6], [6.5, 0, 0]])


def test_log_probabilities_by_hand():
    x = np.array([[0.0, math.log(3), -np.inf, 0.0], [-np.inf] * 4, [1e30, -1e30, 0, 0]])
    lp, h = O.logprobs(x)
    assert np.allclose(lp[0], [math.log(0.2), math.log(0.6), -np.inf, math.log(0.2)])
    assert np.isclose(h[0], -0.4 * math.log(0.2) - 0.6 * math.log(0.6))
    assert np.all(lp[1] == -np.inf) and h[1] == 0 and lp[2, 0] == 0 and h[2] == 0
    flat, h = O.logprobs(np.full((1, 8), 5.0), 0.3)
    assert np.allclose(flat, -math.log(8)) and np.isclose(h[0], math.log(8))
    assert np.array_equal(O.top(x, 4), [[1, 0, 3, -1], [-1] * 4, [0, 2, 3, 1]])
