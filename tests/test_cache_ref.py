"""The fp64 references of cached states and drafted tokens against closed forms,
differences and planted mistakes (no GPU)."""
import numpy as np
import pytest
import torch

import cache_ref as C
from layer_ref import U


def test_numbers_are_the_formats():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(C.NUMBERS["fp8"], bits) and C.NUMBERS["fp8"][-1] == 448
    assert list(C.NUMBERS["fp4"]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and C.NUMBERS["int8"][-1] == 127 / 64


@pytest.mark.parametrize("fmt", ["fp8", "int8", "fp4"])
def test_quantise_rounds_to_the_nearest_once(fmt):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 100)) * np.exp(3 * rng.standard_normal((40, 1)))
    code, sc = C.quantise(x, fmt)
    y = C.dequantise(C.pack(code, fmt), sc, fmt, 100)
    scale = np.repeat(2.0 ** (sc.astype(float) - 127), 32, 1)[:, :100]
    top = C.NUMBERS[fmt][-1]
    assert np.all(np.abs(x) <= top * scale)
    grid = np.concatenate((-C.NUMBERS[fmt][::-1], C.NUMBERS[fmt]))
    best = np.abs(x[..., None] / scale[..., None] - grid).min(-1)
    assert np.allclose(np.abs(x - y) / scale, best, rtol=0, atol=1e-12)
    # half the scale would not hold the block
    for r in range(40):
        for b in range(4):
            block = np.abs(x[r, 32 * b:32 * b + 32]).max()
            assert block > top * 2.0 ** (float(sc[r, b]) - 128)


@pytest.mark.parametrize("fmt,pairs", [("int8", {0.5 / 64: 0, 1.5 / 64: 2, 2.5 / 64: 2}),
                                       ("fp4", {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6})])
def test_ties_go_to_the_even_code(fmt, pairs):
    x = np.zeros((1, 32))
    x[0, 0] = C.NUMBERS[fmt][-1]
    for i, v in enumerate(pairs):
        x[0, i + 1] = v
    code, sc = C.quantise(x, fmt)
    assert sc[0, 0] == 127 and [int(c) for c in code[0, 1:1 + len(pairs)]] == list(pairs.values())


def test_rotation_and_norm_in_closed_form():
    x = np.random.default_rng(1).standard_normal((3, 2, 8))
    angle = np.full((3, 4), np.pi / 2)
    y, _ = C.turn(x, np.zeros_like(x), angle, 8, False)
    assert np.allclose(y, np.concatenate((-x[..., 4:], x[..., :4]), -1))
    y, _ = C.turn(x, np.zeros_like(x), angle, 8, True)
    assert np.allclose(y[..., 0::2], -x[..., 1::2]) and np.allclose(y[..., 1::2], x[..., 0::2])
    out, _ = C.qknorm(x, None, "l2", 0.0, 1.0, angle[:, :2], 4, True)
    assert np.allclose((out ** 2).sum(-1), 1.0)
    out, _ = C.qknorm(x, None, "rms", 0.0, 2.0, angle, 8, False)
    assert np.allclose((out ** 2).mean(-1), 4.0)


@pytest.mark.parametrize("norm", ["l2", "rms", "none"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(norm, interleaved):
    rng = np.random.default_rng(2)
    x, dout, w = rng.standard_normal((3, 2, 10)), rng.standard_normal((3, 2, 10)), 1 + 0.2 * rng.standard_normal(10)
    angle = C.angles(rng.integers(0, 50, (2, 3)), np.array([1.0, 0.3, 0.01]), [0, 1, 0])
    f = lambda x, w: (C.qknorm(x, w, norm, 1e-3, 0.7, angle, 6, interleaved)[0] * dout).sum()     # noqa: E731
    dx, _, dw, _ = C.qknorm_backward(x, w, norm, 1e-3, 0.7, angle, 6, interleaved, dout)
    h = 1e-6
    for got, arr, of in ((dx, x, lambda p: f(p, w)), (dw, w, lambda p: f(x, p))):
        for i in np.ndindex(arr.shape):
            a, b = arr.copy(), arr.copy()
            a[i] += h
            b[i] -= h
            assert abs((of(a) - of(b)) / (2 * h) - got[i]) < 1e-7


def test_decode_is_the_product_form():
    rng = np.random.default_rng(3)
    t = 3
    q, k, v = (rng.standard_normal((t, C.D)) for _ in range(3))
    k /= np.linalg.norm(k, axis=1, keepdims=True)
    g, beta, S = -rng.random((t, C.D)), rng.random(t), rng.standard_normal((C.D, C.D))
    out, end, _, _ = C.decode(q, k, v, g, beta, S)
    for i in range(t):
        S = (np.eye(C.D) - beta[i] * np.outer(k[i], k[i])) @ (np.exp(g[i])[:, None] * S) + beta[i] * np.outer(k[i], v[i])
        assert np.allclose(out[i], S.T @ q[i])
    assert np.allclose(end, S)


def test_verification_keeps_the_targets_distribution():
    """Drafts from q, verified against p: accepted or replaced, the token is distributed as p."""
    rng = np.random.default_rng(4)
    p, q = np.array([0.5, 0.2, 0.0, 0.3]), np.array([0.1, 0.4, 0.2, 0.3])
    n = 40000
    draws = rng.choice(4, n, p=q)
    accept, sample = rng.random(n), rng.random(n)
    seen = np.zeros(4)
    for i in range(n):
        counts, nexts = C.verify(np.array([p, p]), np.array([q, q]), [0, draws[i]], [0, 2], [0, accept[i]], [sample[i]])
        seen[draws[i] if counts[0] == 2 else nexts[0]] += 1
    # a share of n draws has a deviation of at most 1 / (2 sqrt n): four of them
    assert np.all(np.abs(seen / n - p) < 4 / (2 * np.sqrt(n))), seen / n


def test_verification_in_small():
    t = np.array([[0.25, 0.25, 0.5, 0], [0, 1.0, 0, 0], [0.5, 0, 0, 0.5]])
    d = np.array([[9, 9, 9, 9], [0.5, 0.25, 0.25, 0], [0, 1.0, 0, 0]])
    V = lambda *a: C.verify(*a)                                                                   # noqa: E731
    assert V(t, d, [7, 2, 1], [0, 3], [0, .9, .9], [.0]) == ([3], [0])      # all accepted: the last row
    assert V(t, d, [7, 2, 1], [0, 3], [0, .9, .9], [.5]) == ([3], [3])      # 0.5 is not above half of it
    assert V(t, d, [7, 0, 1], [0, 3], [0, .5, 0], [.9]) == ([1], [2])       # 0.5 * 0.5 is not below 0.25
    assert V(t, d, [7, 0, 1], [0, 3], [0, .49, 0], [.9]) == ([3], [3])
    assert V(t, None, [7, 2, 0], [0, 3], [0, .4, 0], [.3]) == ([2], [1])
    assert V(t, None, [7, 2, 1], [0, 3], [0, .5, 0], [.0]) == ([1], [0])    # 0.5 is not below 0.5
    assert V(t, d, [7, 9, -1], [0, 0, 3], [0, 0, 0], [.5, .1]) == ([0, 1], [-1, 2])
    assert V(t * 0, d, [7, 1, 1], [0, 3], [0, 0, 0], [.5]) == ([1], [-1])
    assert V(t, t[[0, 0, 1]], [7, 3, 1], [0, 3], [0, 0, 0], [.5]) == ([1], [2])   # nothing is left of p - q: p itself


def test_planted_mistakes_leave_the_bounds():
    rng = np.random.default_rng(5)
    x, dout = rng.standard_normal((4, 3, 64)), rng.standard_normal((4, 3, 64))
    angle = C.angles(np.arange(4), 0.5 ** np.arange(16), None)
    y, e = C.qknorm(x, None, "l2", 1e-6, 1.0, angle, 32, False)
    for other in (C.qknorm(x, None, "rms", 1e-6, 1.0, angle, 32, False)[0],
                  C.qknorm(x, None, "l2", 1e-6, 1.0, -angle, 32, False)[0],
                  C.qknorm(x, None, "l2", 1e-6, 1.0, angle, 32, True)[0],
                  C.qknorm(x, None, "l2", 1e-4, 1.0, angle, 32, False)[0] * (1 + 1e-4)):
        assert np.any(np.abs(other - y) > 20 * e)
    dx, edx, dw, edw = C.qknorm_backward(x, np.ones(64), "l2", 1e-6, 1.0, angle, 32, False, dout)
    wrong, _, _, _ = C.qknorm_backward(x, np.ones(64), "none", 1e-6, 1.0, angle, 32, False, dout)
    inv, _ = C.inverse(x, "l2", 1e-6)
    assert np.any(np.abs(wrong * inv - dx) > 20 * edx)                    # the part along x left out
    q, k, v = (rng.standard_normal((2, C.D)) for _ in range(3))
    g, beta, S = -rng.random((2, C.D)), rng.random(2), rng.standard_normal((C.D, C.D))
    out, end, eo, es = C.decode(q, 0.1 * k, v, g, beta, S)
    assert eo.max() < 1e-2 and es.max() < 1e-2 and U < 1e-7
    for mistake in (dict(g=-g), dict(beta=beta * (1 + 1e-3)), dict(state=S.T)):
        a = dict(q=q, k=0.1 * k, v=v, g=g, beta=beta, state=S)
        a.update(mistake)
        o, s, _, _ = C.decode(**a)
        assert np.any(np.abs(o - out) > 4 * eo) and np.any(np.abs(s - end) > 4 * es)
