"""The fp64 references of the block operators against their own definitions: gradients
against differences of the forward, special cases against closed forms (CPU)."""
import numpy as np
import pytest

import block_reference as ref


def difference(f, args, k, i, weight, h=1e-6):
    """Central difference of sum(weight * f(args)) along element i of args[k]."""
    out = []
    for s in (h, -h):
        a = [np.array(x, np.float64) if x is not None else None for x in args]
        a[k].reshape(-1)[i] += s
        out.append(sum(float((w * y).sum()) for w, y in zip(weight, f(*a))))
    return (out[0] - out[1]) / (2 * h)


@pytest.mark.parametrize("d", [1, 5, 32])
def test_norm_gradients_are_differences(d):
    rng = np.random.default_rng(d)
    r, w, dy = rng.standard_normal((3, d)), rng.standard_normal(d), rng.standard_normal((3, d))
    dres = rng.standard_normal((3, d))
    dr, dw = ref.norm_bwd(r, w, dy, dres, 1e-3)
    for k, grad in ((0, dr - dres), (1, dw)):
        for i in range(grad.size):
            got = difference(lambda a, b: (ref.norm_fwd(a, b, 1e-3),), (r, w), k, i, (dy,))
            assert abs(got - grad.reshape(-1)[i]) <= 1e-7 * (1 + abs(got))


def test_norm_of_equal_values_is_the_weight():
    w = np.array([1.0, -2.0, 0.5])
    assert np.allclose(ref.norm_fwd(np.full((2, 3), 7.0), w, 0.0), w, atol=1e-15)
    assert np.array_equal(ref.norm_fwd(np.zeros((1, 3)), w, 1e-5), np.zeros((1, 3)))


def test_group_scales():
    y = np.arange(-10.0, 11.0)[None]
    scale, wide = ref.quantise_groups(y, 8)
    assert np.allclose(scale * 448, [[10, 5, 10]]) and wide.shape == y.shape
    assert np.allclose(ref.quantise_groups(y, 0)[0] * 448, [[10]])


@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("W", [2, 4])
def test_conv_gradients_are_differences(W, act):
    rng = np.random.default_rng(W)
    start = [0, 3, 3, 4, 9]                       # lengths 3, 0, 1, 5
    spans = ref.sequences(4, 5, start)
    x, w, bias = rng.standard_normal((9, 3)), rng.standard_normal((3, W)), rng.standard_normal(3)
    state, dy, df = rng.standard_normal((4, W - 1, 3)), rng.standard_normal((9, 3)), rng.standard_normal((4, W - 1, 3))
    g = ref.conv_bwd(x, w, bias, state, spans, act, dy, df)
    for k, name in enumerate(("x", "weight", "bias", "state")):
        for i in range(g[name].size):
            got = difference(lambda a, b, c, d: ref.conv_fwd(a, b, c, d, spans, act)[:2], (x, w, bias, state), k, i,
                             (dy, df))
            assert abs(got - g[name].reshape(-1)[i]) <= 1e-7 * (1 + abs(got)), (name, i)


def test_conv_of_an_impulse_is_its_taps():
    w = np.array([[0.5, -1.0, 2.0, 3.0]])
    x = np.zeros((6, 1))
    x[1] = 1
    y, final, _ = ref.conv_fwd(x, w, None, np.zeros((1, 3, 1)), [(0, 6)], False)
    assert np.array_equal(y[:, 0], [0, 3, 2, -1, 0.5, 0]) and np.array_equal(final[0], x[3:])


def _scan_case(rng, gate, softplus):
    start = [0, 3, 3, 4, 7]
    D, G, N = 4, 2, 3
    c = {"x": rng.standard_normal((7, D)), "dt": rng.standard_normal((7, D)) - (0 if softplus else -1.5),
         "z": rng.standard_normal((7, D)) if gate else None, "A": -np.exp(rng.standard_normal((D, N))),
         "B": rng.standard_normal((7, G, N)), "C": rng.standard_normal((7, G, N)), "D": rng.standard_normal(D),
         "dt_bias": rng.standard_normal(D), "h": rng.standard_normal((4, D, N)), "spans": ref.sequences(4, 3, start),
         "softplus": softplus}
    return c


@pytest.mark.parametrize("gate,softplus", [(True, 1), (False, 0)])
def test_scan_gradients_are_differences(gate, softplus):
    rng = np.random.default_rng(3 + softplus)
    c = _scan_case(rng, gate, softplus)
    dy, dh = rng.standard_normal((7, 4)), rng.standard_normal((4, 4, 3))
    got = ref.scan(c, dy, dh)
    names = [k for k in ("x", "dt", "z", "A", "B", "C", "D", "dt_bias", "h") if c[k] is not None]

    def f(*args):
        out = ref.scan(dict(c, **dict(zip(names, args))))
        return out["y"][0], out["h_final"][0]

    for k, name in enumerate(names):
        grad, bound = got["grad_" + name]
        assert np.all(bound >= 0)
        for i in range(grad.size):
            d = difference(f, [c[n] for n in names], k, i, (dy, dh))
            assert abs(d - grad.reshape(-1)[i]) <= 2e-7 * (1 + abs(d)), (name, i)


def test_scan_without_decay_is_a_running_sum():
    rng = np.random.default_rng(8)
    c = _scan_case(rng, False, 0)
    c.update(A=np.zeros((4, 3)), D=None, dt_bias=None, dt=np.ones((7, 4)), C=np.ones((7, 2, 3)), B=np.ones((7, 2, 3)),
             h=None)
    y = ref.scan(c)["y"][0]
    for lo, hi in c["spans"]:
        assert np.allclose(y[lo:hi], 3 * np.cumsum(c["x"][lo:hi], 0), atol=1e-12)


def test_scan_with_full_forgetting_keeps_one_row():
    rng = np.random.default_rng(9)
    c = _scan_case(rng, False, 0)
    c.update(A=np.full((4, 3), -1e4), dt=np.full((7, 4), 1.0), dt_bias=None, h=None)
    y = ref.scan(c)["y"][0]
    for t in range(7):
        bc = (c["B"][t] * c["C"][t]).sum(1).repeat(2)
        assert np.allclose(y[t], c["x"][t] * (bc + c["D"]), atol=1e-12)
