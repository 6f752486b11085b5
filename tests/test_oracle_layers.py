"""The oracles of the layers beside the scan: against what their formulas fix and against differences."""
import numpy as np
import pytest

from oracle import layers

RNG = np.random.default_rng


def _delta_case(seed, Bt=2, L=7, Hk=2, H=4, N=5, P=3):
    r = RNG(seed)
    k = r.normal(size=(Bt, L, Hk, N))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=r.normal(size=(Bt, L, Hk, N)), k=k, v=r.normal(size=(Bt, L, H, P)), g=-r.uniform(0, 1, (Bt, L, H)),
                beta=r.uniform(0, 1, (Bt, L, H)), h0=r.normal(size=(Bt, H, N, P)))


def test_a_full_write_is_read_back():
    # beta 1 and a unit key: the state answers that key with the value just written
    c = _delta_case(0, Hk=4)
    c["beta"][:] = 1
    c["q"] = c["k"]
    y, _ = layers.delta(**c)
    np.testing.assert_allclose(y, c["v"], atol=1e-12)


def test_no_writes_fade_the_state():
    c = _delta_case(1)
    c["beta"][:] = 0
    _, h = layers.delta(**c)
    np.testing.assert_allclose(h, c["h0"] * np.exp(c["g"].sum(1))[:, :, None, None], rtol=1e-12)


def test_lengths_cut_the_sequences():
    c = _delta_case(2)
    y, h = layers.delta(**c, lengths=np.array([3, 0]))
    short = {n: x[:, :3] if n != "h0" else x for n, x in c.items()}
    y3, h3 = layers.delta(**short)
    np.testing.assert_array_equal(y[0, :3], y3[0])
    np.testing.assert_array_equal(h[0], h3[0])
    assert not y[0, 3:].any() and not y[1].any()
    np.testing.assert_array_equal(h[1], c["h0"][1])


@pytest.mark.parametrize("lengths", [None, [5, 2]])
def test_delta_gradients_against_differences(lengths):
    c = _delta_case(3)
    lengths = None if lengths is None else np.array(lengths)
    r = RNG(4)
    dy, dh = r.normal(size=c["v"].shape), r.normal(size=c["h0"].shape)

    def loss(x):
        y, h = layers.delta(**x, scale=0.7, lengths=lengths)
        return (y * dy).sum() + (h * dh).sum()

    got = layers.delta_backward(**c, scale=0.7, lengths=lengths, dy=dy, dh_final=dh)
    for n in ("q", "k", "v", "g", "beta", "h0"):
        way = r.normal(size=c[n].shape)
        up, down = (loss({**c, n: c[n] + s * 1e-6 * way}) for s in (1, -1))
        assert abs((up - down) / 2e-6 - (got["d" + n] * way).sum()) < 1e-7 * (1 + abs(up)), n


@pytest.mark.parametrize("mode", ["rms", "l2"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_against_differences_and_size(mode, interleaved):
    r = RNG(5)
    x, w, dy = r.normal(size=(2, 3, 2, 10)), r.normal(size=10), r.normal(size=(2, 3, 2, 10))
    f, pos = np.array([1.0, 0.3, 0.01]), r.integers(0, 9, (2, 3))
    args = (f, pos, 1e-3, mode, interleaved)
    dx, dw = layers.qk_norm_backward(x, w, *args, dy)
    for n, d in (("x", dx), ("w", dw)):
        way = r.normal(size=d.shape)

        def loss(s):
            return (layers.qk_norm(x + (s * way if n == "x" else 0), w + (s * way if n == "w" else 0), *args) * dy).sum()

        assert abs((loss(1e-6) - loss(-1e-6)) / 2e-6 - (d * way).sum()) < 1e-7
    y = layers.qk_norm(x, None, f, pos, 0.0, mode, interleaved)  # a rotation keeps the size
    np.testing.assert_allclose((y * y).sum(-1), 10.0 if mode == "rms" else 1.0, rtol=1e-12)
