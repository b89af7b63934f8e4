"""The fp64 references of the layer operators against facts other than
themselves: closed forms, and finite differences of the forward definitions.
These run on a CPU-only host."""
import numpy as np
import pytest

import layer_ref as R

CU = [0, 5, 5, 6, 11]


def _rng(seed=0):
    return np.random.default_rng(seed)


def _slopes(loss, v, eps=1e-6):
    d = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        up, down = v.copy(), v.copy()
        up[i] += eps
        down[i] -= eps
        d[i] = (loss(up) - loss(down)) / (2 * eps)
    return d


def test_scan_closed_forms():
    # no decay: cumulative sums in every sequence; full decay: the inputs
    x = _rng().normal(size=(11, 3))
    init = _rng(1).normal(size=(4, 3))
    f = R.scan(x, np.zeros_like(x), init, CU)
    assert np.allclose(f["h"][:5], init[0] + np.cumsum(x[:5], 0)) and np.allclose(f["h"][6:], init[3] + np.cumsum(x[6:], 0))
    assert np.allclose(f["final"][1], init[1]) and np.allclose(f["final"][0], f["h"][4])
    assert np.allclose(R.scan(x, np.full_like(x, -np.inf), init, CU)["h"], x)


def test_scan_gradients_are_slopes():
    r = _rng(2)
    x, g, init = r.normal(size=(11, 2)), -r.random((11, 2)), r.normal(size=(4, 2))
    do, df = r.normal(size=(11, 2)), r.normal(size=(4, 2))

    def loss(x=x, g=g, init=init):
        f = R.scan(x, g, init, CU)
        return (f["h"] * do).sum() + (f["final"] * df).sum()

    b = R.scan_backward(x, g, init, CU, do, df)
    assert np.allclose(b["dx"], _slopes(lambda v: loss(x=v), x), atol=1e-7)
    assert np.allclose(b["dg"], _slopes(lambda v: loss(g=v), g), atol=1e-7)
    assert np.allclose(b["dinit"], _slopes(lambda v: loss(init=v), init), atol=1e-7)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradients_are_slopes(W, silu):
    r = _rng(3)
    x, w, b, init = r.normal(size=(11, 2)), r.normal(size=(2, W)), r.normal(size=2), r.normal(size=(4, W - 1, 2))
    do, df = r.normal(size=(11, 2)), r.normal(size=(4, W - 1, 2))

    def loss(x=x, w=w, b=b, init=init):
        f = R.conv(x, w, b, init, CU, silu)
        return (f["out"] * do).sum() + (f["final"] * df).sum()

    g = R.conv_backward(x, w, b, init, CU, silu, do, df)
    assert np.allclose(g["dx"], _slopes(lambda v: loss(x=v), x), atol=1e-7)
    assert np.allclose(g["dweight"], _slopes(lambda v: loss(w=v), w), atol=1e-7)
    assert np.allclose(g["dbias"], _slopes(lambda v: loss(b=v), b), atol=1e-7)
    assert np.allclose(g["dinit"], _slopes(lambda v: loss(init=v), init), atol=1e-7)


def test_conv_is_numpy_convolve_and_a_short_sequence_keeps_old_inputs():
    r = _rng(4)
    x, w, init = r.normal(size=(11, 1)), r.normal(size=(1, 4)), r.normal(size=(4, 3, 1))
    f = R.conv(x, w, None, None, [0, 11], False)
    assert np.allclose(f["out"][:, 0], np.convolve(x[:, 0], w[0, ::-1])[:11])
    f = R.conv(x, w, None, init, CU, False)
    assert np.allclose(f["final"][2], [init[2, 1], init[2, 2], x[5]]) and np.allclose(f["final"][1], init[1])


def test_norm_gradients_are_slopes_and_rows_have_unit_size():
    r = _rng(5)
    x, w, do, dr = r.normal(size=(3, 5)), r.normal(size=5), r.normal(size=(3, 5)), r.normal(size=(3, 5))
    assert np.allclose((R.rmsnorm(x, None, None, 0.0)["y"] ** 2).mean(1), 1.0)
    loss = lambda x=x, w=w: (R.rmsnorm(x, None, w, 1e-3)["y"] * do).sum() + (x * dr).sum()   # noqa: E731
    g = R.rmsnorm_backward(x, w, do, dr, 1e-3)
    assert np.allclose(g["dx"], _slopes(lambda v: loss(x=v), x), atol=1e-7)
    assert np.allclose(g["dweight"], _slopes(lambda v: loss(w=v), w), atol=1e-7)


def test_a_wrong_result_is_outside_the_bounds():
    # a rounding of the state to 16 bits between two tokens, and a gate applied one token late
    r = _rng(6)
    x, g = r.normal(size=(40, 4)), -0.1 * r.random((40, 4))
    f = R.scan(x, g, None, [0, 40])
    R.close(f["h"].astype(np.float32), f["h"], f["e_h"], "fp32", "itself")
    bad = f["h"].copy()
    bad[20:] = R.scan(x[20:], g[20:], (f["h"][19:20] * (1 + 2.0 ** -9)), [0, 20])["h"]
    for wrong in (bad, R.scan(x, np.roll(g, 1, 0), None, [0, 40])["h"]):
        with pytest.raises(AssertionError):
            R.close(wrong, f["h"], f["e_h"], "fp32", "planted mistake")
