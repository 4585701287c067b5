"""Pins of the layer operators' oracle (CPU): worked values, invariants, and
gradients against central differences in float64."""
import numpy as np
import pytest

from oracle import layer_oracle as L


def _diff(f, x, h=1e-6):
    """Central differences of the scalar f at x, entry by entry."""
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * h)
    return g


def test_rotary_by_hand():
    x = np.array([[[[1.0, 2.0, 3.0, 4.0, 5.0]]]])
    inv = np.array([np.pi / 2, np.pi])
    pos = np.array([[1]])
    # pairs (0, 2) by 90 degrees, (1, 3) by 180; column 4 copied
    assert np.allclose(L.rotary(x, pos, inv), [[[[-3, -2, 1, -4, 5]]]])
    assert np.allclose(L.rotary(x, pos, inv, interleaved=True), [[[[-2, 1, -3, -4, 5]]]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_inverse_and_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    inv, _ = L.rotary_frequencies(8)
    x, y = rng.normal(size=(2, 1, 1, 1, 10))
    p = np.array([[123456]])
    r = L.rotary(x, p, inv, 1.25, interleaved)
    assert np.allclose(L.rotary(r, p, inv, 1.0, interleaved, inverse=True)[..., :8],
                       1.25 * x[..., :8], atol=1e-9)
    dots = [np.sum(L.rotary(x, np.array([[a]]), inv, 1.0, interleaved) *
                   L.rotary(y, np.array([[a + 5]]), inv, 1.0, interleaved)) for a in (0, 7, 900)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_linear_two_tokens_by_hand():
    q = np.array([[[1.0, 0.0], [1.0, 2.0]]])
    k = np.array([[[2.0, 1.0], [0.0, 3.0]]])
    v = np.array([[[1.0], [5.0]]])
    # S1 = [2 1]; S2 = S1/2 + 5 [0 3] = [1 15.5]
    o, S = L.linear_forward(q, k, v, np.array([np.log(0.5)]), scale=2.0)
    assert np.allclose(o, [[[4.0], [64.0]]]) and np.allclose(S, [[[1.0, 15.5]]])


def test_linear_gradients_against_differences():
    rng = np.random.default_rng(1)
    Hk, Hv, n, d = 2, 4, 5, 3
    q, k = rng.normal(size=(2, Hk, n, d))
    v, dO = rng.normal(size=(2, Hv, n, d))
    S0, dS = rng.normal(size=(2, Hv, d, d))
    lg = -rng.uniform(0.05, 1.0, Hv)

    def loss():
        o, S = L.linear_forward(q, k, v, lg, S0, 0.7)
        return (o * dO).sum() + (S * dS).sum()

    for got, x in zip(L.linear_backward(q, k, v, lg, S0, dO, dS, 0.7), (q, k, v, S0)):
        assert np.allclose(got, _diff(loss, x), atol=1e-7)


def test_linear_cut_anywhere_is_the_same():
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(2, 1, 9, 4))
    v = rng.normal(size=(1, 9, 4))
    lg = np.array([-0.2])
    o, S = L.linear_forward(q, k, v, lg)
    o1, S1 = L.linear_forward(q[:, :4], k[:, :4], v[:, :4], lg)
    o2, S2 = L.linear_forward(q[:, 4:], k[:, 4:], v[:, 4:], lg, S1)
    assert np.allclose(np.concatenate([o1, o2], 1), o) and np.allclose(S, S2)


def test_block_norm_by_hand():
    y = np.array([[[3.0, 4.0]]])                       # rms^2 = 12.5
    x, N = L.block_norm(y, np.zeros((1, 2)), np.ones(2), np.array([[1.0, -1.0]]),
                        np.array([2.0, 3.0]), scale=2.0, eps=0.0, act="sigmoid")
    e = np.array([3.0, 4.0]) / np.sqrt(12.5) + [1.0, -1.0]    # the gate is one half
    assert np.allclose(x, e)
    assert np.allclose(N, [2.0, 3.0] * e / np.sqrt((e * e).mean()))


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("parts", ["zprn", "zp", "n", "rn", "z"])
def test_block_norm_gradients_against_differences(act, parts):
    rng = np.random.default_rng(3)
    rows, H, d = 3, 2, 4
    y = rng.normal(size=(rows, H, d))
    z = rng.normal(size=(rows, 8)) if "z" in parts else None
    wo = rng.normal(size=8) if "p" in parts else None
    r = rng.normal(size=(rows, 8)) if "r" in parts else None
    wi = rng.normal(size=8) if "n" in parts else None
    dX, dN = rng.normal(size=(2, rows, 8))

    def loss():
        x, N = L.block_norm(y, z, wo, r, wi, 0.6, 1e-3, act)
        return (x * dX).sum() + (0.0 if N is None else (N * dN).sum())

    got = L.block_norm_backward(y, z, wo, r, wi, dX, dN, 0.6, 1e-3, act)
    for g, x in zip(got, (y, z, r, wo, wi)):
        assert (g is None) == (x is None)
        if x is not None:
            assert np.allclose(g, _diff(loss, x), atol=1e-7)
