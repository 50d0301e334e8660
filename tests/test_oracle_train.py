"""The float64 oracle of the norm and the router's training side against
central differences and closed forms."""
import numpy as np
import pytest

from oracle import route as oroute
from oracle import train as otrain


def _diff(f, x, eps=1e-6):
    """Gradient of scalar f at x by central differences."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        old = x[i]
        x[i] = old + eps
        a = f()
        x[i] = old - eps
        b = f()
        x[i] = old
        g[i] = (a - b) / (2 * eps)
    return g


def test_e4m3_table():
    v = otrain.e4m3_values()
    assert len(v) == 127 and v[0] == 0 and v[1] == 2.0 ** -9 and v[-1] == 448.0 and v[0x38] == 1.0
    assert np.all(np.diff(v) > 0)


def test_mx8_round_trip_and_scale_rule():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((5, 64)) * np.exp(rng.uniform(-20, 20, (5, 1)))
    v[4] = 0.0
    codes, scales = otrain.mx8_encode(v)
    back = otrain.mx8_decode(codes, scales)
    amax = np.abs(v.reshape(5, 2, 32)).max(2)
    e = scales.astype(int) - 127
    assert np.all(amax <= 448 * 2.0 ** e)
    assert np.all((amax > 448 * 2.0 ** (e - 1)) | (e == -127))
    # half a step of e4m3 (2^-4 relative), or half its least step times the scale
    bound = np.maximum(np.abs(v) * 2.0 ** -4, np.repeat(2.0 ** (e - 10.0), 32, 1))
    assert np.all(np.abs(back - v) <= bound)
    assert np.all(scales[4] == 0) and np.all(codes[4] == 0)
    # exactly 448 2^e stays in range, the next value up takes the next scale
    w = np.zeros((2, 32))
    w[0, 3], w[1, 3] = 448.0, np.nextafter(448.0, 1e9)
    c, s = otrain.mx8_encode(w)
    assert s[0, 0] == 127 and s[1, 0] == 128 and c[0, 3] == 0x7E and c[1, 3] == 0x76
    w[0, 5] = np.inf
    c, s = otrain.mx8_encode(w)
    assert s[0, 0] == 255 and np.all(np.isnan(otrain.mx8_decode(c, s)[0]))


def test_norm_gradients_by_differences():
    rng = np.random.default_rng(2)
    T, H = 3, 8
    h, w, c, d = (rng.standard_normal(s) for s in ((T, H), (H,), (T, H), (T, H)))
    eps = 1e-3

    def f():
        r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
        return (c * h * r * w).sum() + (d * h).sum()

    r = 1 / np.sqrt((h * h).mean(1) + eps)
    dx, dw = otrain.rms_norm_backward(c, d, h * r[:, None], r, w)
    assert np.allclose(dx, _diff(f, h), atol=1e-8)
    assert np.allclose(dw, _diff(f, w), atol=1e-8)


@pytest.mark.parametrize("offsets,mask", [(None, False), ([0, 2, 2, 6], True)])
def test_balance_gradient_by_differences(offsets, mask):
    rng = np.random.default_rng(3)
    T, E, k = 7, 5, 2
    z = rng.standard_normal((T, E))
    z[1, 2] = -np.inf
    ids = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    m = None if not mask else np.array([1, 1, 0, 1, 1, 1, 1])
    got = otrain.balance_loss(z, ids, E, k, 0.3, m, offsets)
    fin = z.copy()
    zz = np.where(np.isneginf(z), -40.0, z)   # e^-40: the differences see the same function
    f = lambda: otrain.balance_loss(zz, ids, E, k, 0.3, m, offsets)["loss"]  # noqa: E731
    assert np.allclose(got["dlogits"], _diff(f, zz), atol=1e-9)
    assert np.array_equal(fin, z)
    n = got["n_valid"]
    assert n[:-1].sum() * k == got["counts"].sum() and n[-1] == (n[:-1] > 0).sum()


def test_balance_loss_uniform_is_alpha():
    """Equal probabilities and equal counts: sum_e 1 * (1/E) = 1, loss alpha."""
    E, k, T = 4, 2, 6
    ids = np.array([[0, 1], [2, 3], [0, 1], [2, 3], [0, 2], [1, 3]], np.int32)
    got = otrain.balance_loss(np.zeros((T, E)), ids, E, k, 0.01)
    assert abs(got["loss"] - 0.01) < 1e-15


@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradients_by_differences(renorm):
    rng = np.random.default_rng(4)
    T, H, E, k = 4, 6, 7, 3
    x, wr, b = rng.standard_normal((T, H)), rng.standard_normal((E, H)), rng.standard_normal(E)
    cw, cz = rng.standard_normal((T, k)), rng.standard_normal((T, E))
    ids = oroute.select_topk(x @ wr.T + b, k)

    def f():
        z = x @ wr.T + b
        return (cw * oroute.topk_weights(z, ids, renorm)).sum() + (cz * z).sum()

    z = x @ wr.T + b
    dz = otrain.route_dlogits(z, ids, oroute.topk_weights(z, ids, renorm), cw, renorm, cz, E)
    dx, dwr, db = otrain.route_backward(dz, x, wr)
    assert np.allclose(dx, _diff(f, x), atol=1e-7)
    assert np.allclose(dwr, _diff(f, wr), atol=1e-7)
    assert np.allclose(db, _diff(f, b), atol=1e-7)


def test_route_gradient_of_dropped_and_repeated_ids():
    """An id outside [0, E) passes nothing; an id listed twice gets both."""
    w = np.array([[0.5, 0.3, 0.2]])
    d = np.array([[1.0, 2.0, 3.0]])
    dz = otrain.route_dlogits(None, np.array([[1, -1, 1]]), w, d, True, None, 3)
    dot = 0.5 * 1 + 0.2 * 3
    assert np.allclose(dz, [[0, 0.5 * (1 - dot) + 0.2 * (3 - dot), 0]])
