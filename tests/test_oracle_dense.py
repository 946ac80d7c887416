"""The float64 forms of the exact-attention operators: gradients against
finite differences, degenerate masks, rotary identities, and the frequencies
that the binding computes.  CPU only."""
import math

import numpy as np
import pytest

from oracle import dense_ref
from structured_sub_quadratic_b200 import api


@pytest.mark.parametrize("causal,lens", [(False, None), (True, None), (True, [5, 0])])
def test_gradients_match_differences(causal, lens):
    r = np.random.default_rng(0)
    q, do = r.standard_normal((2, 2, 4, 4, 3))
    k, v = r.standard_normal((2, 2, 2, 6, 3))
    grads = dense_ref.dense_backward(q, k, v, do, causal, lens)
    f = lambda *x: (dense_ref.dense_forward(*x, causal, lens)[0] * do).sum()  # noqa: E731
    h = 1e-6
    for a, g in enumerate(grads):
        for at in [(0, 0, 0, 0), (0, 1, 3, 2), (1, 0, 2, 1), (1, 1, 1, 0), (0, 0, 3, 1)]:
            x = [t.copy() for t in (q, k, v)]
            y = [t.copy() for t in (q, k, v)]
            x[a][at] += h
            y[a][at] -= h
            # central difference: h^2 and 1e-16 / h, both below 1e-9
            assert abs((f(*x) - f(*y)) / (2 * h) - g[at]) < 1e-8


def test_rows_without_keys():
    r = np.random.default_rng(1)
    q, k, v = (r.standard_normal((1, 1, n, 4)) for n in (5, 3, 3))
    o, lse = dense_ref.dense_forward(q, k, v, causal=True)
    assert (o[0, 0, :2] == 0).all() and np.isneginf(lse[0, 0, :2]).all()
    assert np.allclose(o[0, 0, 2], v[0, 0, 0]) and np.isfinite(lse[0, 0, 2:]).all()


def test_decode_is_the_last_row():
    r = np.random.default_rng(2)
    q = r.standard_normal((2, 4, 1, 8))
    k, v = r.standard_normal((2, 2, 2, 7, 8))
    o, lse = dense_ref.dense_forward(q, k, v, lens=[7, 4])
    pages = [x.reshape(2, 2, 7, 8) for x in (k, v)]  # one page of seven rows per sequence
    O, L, _ = dense_ref.decode(q[:, :, 0], *pages, np.array([[0], [1]]), [7, 4])
    assert np.allclose(O, o[:, :, 0]) and np.allclose(L, lse[..., 0])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_keeps_products_of_equal_distances(interleaved):
    r = np.random.default_rng(3)
    q, k = r.standard_normal((2, 1, 1, 1, 16))
    f, m = api.rotary_frequencies((8, 6))
    dot = []
    for at in (0, 1000):
        p = np.array([[[at + 7], [at + 2]]])
        s = np.array([[[at + 3], [at]]])
        a = dense_ref.rotary(q, p, (8, 6), f, m, interleaved)
        b = dense_ref.rotary(k, s, (8, 6), f, m, interleaved)
        dot.append((a * b).sum())
        back = dense_ref.rotary(a, p, (8, 6), f, m, interleaved, inverse=True)
        assert np.allclose(back, q) and np.array_equal(a[..., 14:], q[..., 14:])
    assert abs(dot[0] - dot[1]) < 1e-9


def test_frequencies():
    f, m = api.rotary_frequencies((8, 4))
    assert np.allclose(f, [1, 0.1, 0.01, 0.001, 1, 0.01]) and m == 1
    assert np.allclose(api.rotary_frequencies((8,), scaling=("linear", 4.0))[0],
                       np.array([1, 0.1, 0.01, 0.001]) / 4)
    ntk = api.rotary_frequencies((8,), scaling=("ntk", 4.0))[0]
    assert ntk[0] == 1 and math.isclose(ntk[3], 0.001 / 4)  # the slowest pair: four-fold
    parts, m = api.rotary_frequencies((64,), scaling=("parts", 4.0, 4096, 1, 32))
    plain = api.rotary_frequencies((64,))[0]
    turns = np.array(plain) * 4096 / (2 * math.pi)
    ratio = np.array(parts) / np.array(plain)
    assert np.allclose(ratio[turns >= 32], 1) and np.allclose(ratio[turns <= 1], 0.25)
    assert (np.diff(ratio) <= 1e-12).all() and math.isclose(m, 0.1 * math.log(4) + 1)
    for bad in (("ntk",), ("linear", 0), ("other", 2.0), ("parts", 2.0, 4096, 32, 1),
                ("parts", 0.5, 4096, 1, 32)):
        with pytest.raises(ValueError):
            api.rotary_frequencies((64,), scaling=bad)
    with pytest.raises(ValueError):
        api.rotary_frequencies((64,), base=0.0)
