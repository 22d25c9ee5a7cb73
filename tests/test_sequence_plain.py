"""The plain float64 scan and convolution that the GPU tests compare with: their cotangents against central differences
of their forward, the scan against the dense solve of its block lower-bidiagonal system, splits against the whole, and
the magnitudes that the tolerances are made of."""
import numpy as np
import pytest

from tests import sequence_plain as plain


def scan_inputs(rng, rows, d, n, groups, gate=True, softplus=True):
    v = dict(x=rng.standard_normal((rows, d)), dt=0.5 * rng.standard_normal((rows, d)),
             A=-np.exp(rng.standard_normal((d, n))), B=rng.standard_normal((rows, groups, n)),
             C=rng.standard_normal((rows, groups, n)), D=rng.standard_normal(d), state=rng.standard_normal((d, n)),
             dt_bias=rng.standard_normal(d) - 1)
    if gate:
        v["z"] = rng.standard_normal((rows, d))
    return v


def differences(f, inputs, key, eps=1e-6):
    """Central differences of the scalar f(inputs) along every entry of one input."""
    out = np.empty_like(inputs[key])
    for i in np.ndindex(out.shape):
        vals = []
        for s in (eps, -eps):
            v = dict(inputs)
            v[key] = inputs[key].copy()
            v[key][i] += s
            vals.append(f(v))
        out[i] = (vals[0] - vals[1]) / (2 * eps)
    return out


@pytest.mark.parametrize("gate", [True, False])
def test_scan_cotangents_are_differences(gate):
    rng = np.random.default_rng(1)
    v = scan_inputs(rng, 5, 4, 3, 2, gate)
    yb, sb = rng.standard_normal((5, 4)), rng.standard_normal((4, 3))

    def loss(w):
        r = plain.scan(**w, softplus=True)
        return (r["y"] * yb).sum() + (r["state"] * sb).sum()

    g = plain.scan(**v, softplus=True, yb=yb, stateb=sb)
    for key in v:
        d = differences(loss, v, key)
        assert np.abs(g[key + "b"] - d).max() <= 1e-7 * (1 + np.abs(d).max()), key


def test_conv_cotangents_are_differences():
    rng = np.random.default_rng(2)
    for rows, k in ((1, 4), (2, 4), (6, 3)):
        v = dict(x=rng.standard_normal((rows, 3)), weight=rng.standard_normal((3, k)), bias=rng.standard_normal(3),
                 state=rng.standard_normal((k - 1, 3)))
        yb, sb = rng.standard_normal((rows, 3)), rng.standard_normal((k - 1, 3))

        def loss(w):
            r = plain.conv(**w, silu=True)
            return (r["y"] * yb).sum() + (r["state"] * sb).sum()

        g = plain.conv(**v, silu=True, yb=yb, stateb=sb)
        for key in v:
            d = differences(loss, v, key)
            assert np.abs(g[key + "b"] - d).max() <= 1e-7 * (1 + np.abs(d).max()), key


def test_scan_is_the_solve_of_a_bidiagonal_system():
    """h = M^-1 u with M_tt = I and M_{t,t-1} = -diag(a_t), one channel at a time."""
    rng = np.random.default_rng(3)
    rows, d, n = 6, 2, 3
    v = scan_inputs(rng, rows, d, n, 1, gate=False)
    v["D"], v["state"] = np.zeros(d), np.zeros((d, n))
    step = np.logaddexp(v["dt"] + v["dt_bias"], 0)
    y = plain.scan(**v, softplus=True)["y"]
    for c in range(d):
        M = np.eye(rows * n)
        for t in range(1, rows):
            M[t * n:(t + 1) * n, (t - 1) * n:t * n] = -np.diag(np.exp(step[t, c] * v["A"][c]))
        h = np.linalg.solve(M, ((step[:, c] * v["x"][:, c])[:, None] * v["B"][:, 0]).ravel()).reshape(rows, n)
        assert np.allclose((h * v["C"][:, 0]).sum(1), y[:, c], atol=1e-12)


def test_splits_equal_the_whole_and_magnitudes_bound():
    rng = np.random.default_rng(4)
    v = scan_inputs(rng, 9, 4, 5, 2)
    whole = plain.scan(**v, softplus=True)
    a = {k: (w[:4] if k in ("x", "dt", "B", "C", "z") else w) for k, w in v.items()}
    b = {k: (w[4:] if k in ("x", "dt", "B", "C", "z") else w) for k, w in v.items()}
    ra = plain.scan(**a, softplus=True)
    rb = plain.scan(**{**b, "state": ra["state"]}, softplus=True)
    assert np.allclose(np.concatenate([ra["y"], rb["y"]]), whole["y"], atol=1e-13)
    assert np.allclose(rb["state"], whole["state"], atol=1e-13)
    yb = rng.standard_normal((9, 4))
    g, m = (plain.scan(**v, softplus=True, yb=yb, mag=q) for q in (False, True))
    for key in g:
        assert (np.abs(g[key]) <= m[key] * (1 + 1e-12)).all(), key
    x, w = rng.standard_normal((7, 3)), rng.standard_normal((3, 4))
    one = plain.conv(x, w, silu=True)
    first = plain.conv(x[:2], w, silu=True)
    rest = plain.conv(x[2:], w, silu=True, state=first["state"])
    assert np.allclose(np.concatenate([first["y"], rest["y"]]), one["y"], atol=1e-14)
    assert np.array_equal(rest["state"], one["state"])
