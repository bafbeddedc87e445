"""The 64-bit references of the layer operators against closed forms and central differences (no GPU)."""
import numpy as np
import pytest

from tests import layers_reference as ref


def _attn(seed, B=2, T=5, H=4, Hk=2, dk=3, dv=2, per_head=False):
    r = np.random.RandomState(seed)
    g = -r.rand(H) if per_head else -r.rand(B, T, H)
    return dict(q=r.randn(B, T, Hk, dk), k=r.randn(B, T, Hk, dk), v=r.randn(B, T, H, dv), g=g,
                S0=r.randn(B, H, dv, dk), lengths=np.array([T, 3][:B])), r


def test_linattn_without_decay_is_a_running_sum():
    a, _ = _attn(0, Hk=4)
    a.update(g=np.zeros(4), S0=None, lengths=None)
    got = ref.linattn(**a)["o"]
    for t in range(5):
        want = sum(np.einsum("bhd,bhd->bh", a["q"][:, t], a["k"][:, j])[..., None] * a["v"][:, j] for j in range(t + 1))
        assert np.allclose(got[:, t], want, rtol=1e-12, atol=1e-12)


def test_linattn_cleared_state_forgets():
    a, _ = _attn(1)
    a["lengths"] = None
    a["g"][:, 2] = -np.inf
    late = {n: (x[:, 2:] if n in "qkvg" else x) for n, x in a.items()}
    late["S0"] = None
    assert np.array_equal(ref.linattn(**a)["o"][:, 2:], ref.linattn(**late)["o"])


@pytest.mark.parametrize("per_head", [False, True])
def test_linattn_gradient_is_the_differences(per_head):
    a, r = _attn(2, per_head=per_head)
    do, dST = r.randn(2, 5, 4, 2), r.randn(2, 4, 2, 3)
    got = ref.linattn(**a, scale=0.7, do=do, dST=dST)

    def loss(**change):
        out = ref.linattn(**{**a, **change}, scale=0.7)
        live = np.arange(5)[None, :] < a["lengths"][:, None]
        return (out["o"] * do * live[..., None, None]).sum() + (out["ST"] * dST).sum()

    for name in ("q", "k", "v", "g", "S0"):
        u, e = r.randn(*a[name].shape), 1e-5
        diff = (loss(**{name: a[name] + e * u}) - loss(**{name: a[name] - e * u})) / (2 * e)
        # truncation e^2 times a third derivative of order 10, rounding 1e-16 |L| / e
        assert abs(diff - (got["d" + name] * u).sum()) <= 1e-8 * max(1.0, abs(diff)), name


def test_rmsnorm_gradient_is_the_differences():
    r = np.random.RandomState(3)
    x, w, dy, dh = r.randn(4, 6), r.randn(6), r.randn(4, 6), r.randn(4, 6)
    y, h, rstd = ref.rmsnorm(x, w)
    dx, dw = ref.rmsnorm_bwd(dy, h, w, rstd, dh)
    loss = lambda x, w: (ref.rmsnorm(x, w)[0] * dy).sum() + (x * dh).sum()  # noqa: E731
    u, s, e = r.randn(4, 6), r.randn(6), 1e-5
    assert abs((loss(x + e * u, w) - loss(x - e * u, w)) / (2 * e) - (dx * u).sum()) <= 1e-8
    assert abs((loss(x, w + e * s) - loss(x, w - e * s)) / (2 * e) - (dw * s).sum()) <= 1e-8


def test_linattn_reference_notices_a_planted_mistake():
    """A decay applied one step late, or a head's key of the wrong group, moves the result by far more than the
    tolerances of the GPU tests."""
    a, _ = _attn(4)
    good = ref.linattn(**a)["o"]
    late = dict(a, g=np.roll(a["g"], 1, axis=1))
    swapped = dict(a, k=a["k"][:, :, ::-1])
    for bad in (late, swapped):
        assert np.abs(ref.linattn(**bad)["o"] - good).max() > 0.05 * np.abs(good).max()
