"""Pins of the gated delta rule's oracle: the Gated DeltaNet-2 oracle under its reduction, a hand
example, associative recall, split and resume, shared heads, and finite differences of the gradients."""
import numpy as np
import pytest

import oracle
from linear_recurrent_token_b200 import inputs


def make(seed=1, **kw):
    base = dict(B=2, HK=2, H=4, T=9, K=6, V=5)
    base.update(kw)
    return inputs.gdr_inputs(dtype="f64", seed=seed, **base)


def args(x, names=("q", "k", "v", "g", "beta")):
    return [x[n] for n in names]


def test_is_the_reduction_of_gdn2():
    x = make(HK=4)
    wide = lambda a, d: np.repeat(a[..., None], d, axis=-1)
    o, S = oracle.gdr_sequential(*args(x), x["S0"])
    o2, S2 = oracle.gdn2_sequential(x["q"], x["k"], x["v"], wide(x["g"], 6), wide(x["beta"], 6), wide(x["beta"], 5),
                                    x["S0"])
    assert np.allclose(o, o2, rtol=1e-13, atol=1e-14) and np.allclose(S, S2, rtol=1e-13, atol=1e-14)


def test_hand_example():
    """K = V = 1: S = 2, e^g = 1/2, k = 1, beta = 1/2, v = 3: S' = 1, S = 1 + (3 - 1) / 2 = 2; q = 4: o = 8."""
    one = lambda x: np.full((1, 1, 1, 1), float(x))
    o, S = oracle.gdr_sequential(one(4), one(1), one(3), np.full((1, 1, 1), np.log(0.5)), np.full((1, 1, 1), 0.5),
                                 one(2))
    assert np.allclose(o, 8) and np.allclose(S, 2)


def test_stores_a_value_under_a_unit_key():
    x = make(HK=4)
    x["beta"][:] = 1.0
    x["q"] = x["k"].copy()  # reading with the key just written
    o, _ = oracle.gdr_sequential(*args(x), x["S0"])
    assert np.allclose(o, x["v"], atol=1e-12)


def test_a_token_without_write_strength_and_decay_is_passed_over():
    x = make()
    o, S = oracle.gdr_sequential(*args(x), x["S0"])
    x2 = {n: np.insert(x[n], 4, 0.0, axis=2) for n in ("g", "beta")}
    x2 |= {n: np.insert(x[n], 4, 7.0, axis=2) for n in ("q", "k", "v")}
    o2, S2 = oracle.gdr_sequential(*args(x2), x["S0"])
    assert np.allclose(np.delete(o2, 4, axis=2), o) and np.allclose(S2, S)


def test_a_token_with_full_decay_forgets():
    x = make()
    x["g"][:, :, 5] = -np.inf
    _, S = oracle.gdr_sequential(*args(x), x["S0"])
    tail = {n: x[n][:, :, 5:] for n in ("q", "k", "v", "g", "beta")}
    _, S2 = oracle.gdr_sequential(*args(tail))
    assert np.allclose(S, S2)


def test_split_and_resume():
    x = make(T=11)
    o, S = oracle.gdr_sequential(*args(x), x["S0"])
    a = {n: x[n][:, :, :4] for n in ("q", "k", "v", "g", "beta")}
    b = {n: x[n][:, :, 4:] for n in ("q", "k", "v", "g", "beta")}
    oa, Sa = oracle.gdr_sequential(*args(a), x["S0"])
    ob, Sb = oracle.gdr_sequential(*args(b), Sa)
    assert np.allclose(np.concatenate([oa, ob], 2), o) and np.allclose(Sb, S)


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "S0"])
def test_gradients_against_differences(name):
    """Central differences of <do, o> + <dS, S_T> along random directions: error O(h^2) ~ 1e-10."""
    x = make(seed=4)
    rng = np.random.default_rng(5)
    do, dS = rng.standard_normal((2, 4, 9, 5)), rng.standard_normal((2, 4, 6, 5))
    grads = oracle.gdr_sequential_backward(*args(x), do, x["S0"], dS)

    def loss(y):
        o, S = oracle.gdr_sequential(*args(y), y["S0"])
        return (o * do).sum() + (S * dS).sum()

    for _ in range(4):
        d = rng.standard_normal(x[name].shape)
        h = 1e-5
        num = (loss({**x, name: x[name] + h * d}) - loss({**x, name: x[name] - h * d})) / (2 * h)
        assert abs(num - (grads["d" + name] * d).sum()) <= 1e-7 * max(1.0, abs(num))


def test_gradient_of_the_gates_where_they_are_zero():
    """beta = 0 still has a gradient (the write that it holds back), and so has a full reset's none."""
    x = make(seed=6)
    x["beta"][:, :, 3] = 0.0
    do, dS = np.ones((2, 4, 9, 5)), np.ones((2, 4, 6, 5))
    d = oracle.gdr_sequential_backward(*args(x), do, x["S0"], dS)
    assert np.abs(d["dbeta"][:, :, 3]).min() > 0 and np.allclose(d["dv"][:, :, 3], 0)
    x["g"][:, :, 3] = -np.inf
    do[:, :, :3] = 0.0  # nothing reads the state before it is reset
    d = oracle.gdr_sequential_backward(*args(x), do, x["S0"], dS)
    assert np.allclose(d["dg"][:, :, 3], 0) and np.allclose(d["dS0"], 0)
