"""The tests' own 64-bit implementations: gradients against central differences of the forward, known values."""
import numpy as np
import pytest

from tests import tokens_reference as ref


@pytest.mark.parametrize("ragged,packed", [(False, False), (True, False), (False, True), (True, True)])
def test_gated_gradients_against_differences(ragged, packed):
    rng = np.random.default_rng(3 + 2 * ragged + packed)
    B, T, D = 2, 7, 3
    a = dict(x=rng.normal(size=(B, T, D)), r=rng.normal(size=(B, T, D)), i=rng.normal(size=(B, T, D)),
             lam=rng.normal(size=D) - 3, h0=rng.normal(size=(B, D)))
    more = dict(lengths=[5, 7] if ragged else None, reset=rng.random((B, T)) < 0.3 if packed else None, rate=3.0)
    dy, dhT = rng.normal(size=(B, T, D)), rng.normal(size=(B, D))

    def loss(v):
        o = ref.gated(**v, **more)
        return (o["y"] * dy).sum() + (o["hT"] * dhT).sum()

    got = ref.gated(**a, **more, dy=dy, dhT=dhT)
    for name in a:
        want = np.zeros_like(a[name])
        for at in np.ndindex(want.shape):
            up, down = ({k: v.copy() for k, v in a.items()} for _ in range(2))
            up[name][at] += 1e-5
            down[name][at] -= 1e-5
            want[at] = (loss(up) - loss(down)) / 2e-5
        # a central difference of step 1e-5 is off by some 1e-10 of second derivatives, and 1e-16 / 1e-5 of the loss
        assert np.abs(got["d" + name] - want).max() < 1e-7 * max(1.0, np.abs(want).max()), name


def test_gated_known_values():
    """Gates at zero (one half), lam so that softplus is log 2: a = 2^-(rate / 2), and the state's variance stays one."""
    one = np.ones((1, 3, 1))
    o = ref.gated(one, 0 * one, 0 * one, np.zeros(1), h0=np.array([[2.0]]), rate=2.0)
    a, b = 0.5, 0.5 * 0.75 ** 0.5
    want, h = [], 2.0
    for _ in range(3):
        h = a * h + b
        want.append(h)
    assert np.allclose(o["y"][0, :, 0], want, rtol=1e-15)


def test_sample_known_values():
    x = np.log([0.1, 0.4, 0.3, 0.2])
    for u, want in ((0.0, 0), (0.09, 0), (0.11, 1), (0.49, 1), (0.51, 2), (0.79, 2), (0.81, 3), (1.0, 3)):
        assert ref.sample(x, u)[0] == want, u
    assert ref.sample(x, 0.0, top_k=2)[0] == 1 and ref.sample(x, 0.58, top_k=2)[0] == 2
    assert ref.sample(x, 0.99, top_p=0.4 - 1e-9)[0] == 1 and ref.sample(x, 0.99, top_p=0.41)[0] == 2
    assert ref.sample(x, 0.99, min_p=0.6)[0] == 2 and ref.sample(x, 0.99, min_p=0.4)[0] == 3
    assert ref.sample(x, 0.9, temperature=0.0)[:2] == (1, 0.0)
    assert ref.sample([-np.inf] * 3, 0.5)[0] == -1 and ref.sample([0.0, np.nan], 0.5)[0] == -1
    assert ref.sample([1.0, 1.0, 1.0, 0.0], 0.99, top_k=2)[0] == 1     # of equals the first by index
    assert ref.sample([0.0, np.inf, 5.0, np.inf], 0.6)[0] == 3


def test_embed_known_values():
    W = np.arange(6.0).reshape(3, 2)
    assert (ref.embed([2, -1, 0, 3], W, 2.0) == [[8, 10], [0, 0], [0, 2], [0, 0]]).all()
    dW, size, many = ref.embed_bwd([1, 1, -1, 0], [[1, 2], [3, -4], [9, 9], [5, 6]], 3, 2.0)
    assert (dW == [[10, 12], [8, -4], [0, 0]]).all() and (size[1] == [8, 12]).all() and (many == [1, 2, 0]).all()
