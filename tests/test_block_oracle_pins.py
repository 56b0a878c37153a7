"""Pins of the oracle for the operators around retention: values worked by
hand, agreement with the retention oracle where the two meet, and gradients
against central differences."""
import math

import numpy as np
import pytest

import oracle

LN3 = math.log(3.0)       # sigmoid(ln 3) = 3/4


def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_scan_by_hand():
    f = np.array([[[LN3], [0.0]]])                      # a = 3/4, 1/2
    x = np.array([[[4.0], [8.0]]])
    y, h = oracle.scan(x, f, "logit", state_in=np.array([[2.0]]))
    assert np.allclose(h[0, :, 0], [0.75 * 2 + 0.25 * 4, 0.5 * 2.5 + 0.5 * 8])
    f = np.log(np.array([[[0.5], [0.25]]]))
    y, h = oracle.scan(x, f, "log", gate=np.full((1, 2, 1), LN3), state_in=np.array([[2.0]]))
    assert np.allclose(h[0, :, 0], [5.0, 9.25])
    assert np.allclose(y, h * 0.75 * LN3)


def test_scan_with_a_fixed_decay_is_retention_with_one_channel():
    """d_k = d_v = 1, q = 1: S_n = gamma S_(n-1) + k_n v_n."""
    H, N = 3, 40
    gam = np.array([0.5, 0.9, 0.97])
    k, v = _rand(1, 1, H, N, 1), _rand(2, 1, H, N, 1)
    o, s = oracle.recurrent(np.ones_like(k), k, v, gam, _rand(3, 1, H, 1, 1))
    x = (k * v)[:, :, :, 0].transpose(0, 2, 1)
    f = np.broadcast_to(np.log(gam), (1, N, H))
    y, h = oracle.scan(x, f, "log", state_in=_rand(3, 1, H, 1, 1)[:, :, 0, 0])
    assert np.allclose(y, o[:, :, :, 0].transpose(0, 2, 1), atol=1e-13)
    assert np.allclose(h[:, -1], s[:, :, 0, 0], atol=1e-13)


@pytest.mark.parametrize("form", ["logit", "log"])
def test_zero_decay_starts_afresh(form):
    f = -np.abs(_rand(4, 2, 9, 5))
    f[:, 4] = -np.inf
    x = _rand(5, 2, 9, 5)
    y, _ = oracle.scan(x, f, form, state_in=_rand(6, 2, 5))
    tail, _ = oracle.scan(x[:, 4:], f[:, 4:], form)
    assert np.array_equal(y[:, 4:], tail)
    _, df, _, ds = oracle.scan_backward(x, f, form, _rand(7, 2, 9, 5), state_in=_rand(6, 2, 5))
    assert np.isfinite(df).all() and not df[:, 4].any()


def _difference(fun, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = fun()
        x[i] = keep - eps
        g[i] = (up - fun()) / (2 * eps)
        x[i] = keep
    return g


@pytest.mark.parametrize("form", ["logit", "log"])
@pytest.mark.parametrize("gated", [False, True])
def test_scan_backward_against_differences(form, gated):
    x, f, g = _rand(1, 2, 6, 3), -np.abs(_rand(2, 2, 6, 3)), _rand(3, 2, 6, 3)
    s0, d_y, d_s = _rand(4, 2, 3), _rand(5, 2, 6, 3), _rand(6, 2, 3)
    gate = g if gated else None

    def loss():
        y, h = oracle.scan(x, f, form, gate, s0)
        return (y * d_y).sum() + (h[:, -1] * d_s).sum()

    dx, df, dg, ds = oracle.scan_backward(x, f, form, d_y, gate, s0, d_s)
    for got, wrt in ((dx, x), (df, f), (ds, s0)) + (((dg, g),) if gated else ()):
        assert np.allclose(got, _difference(loss, wrt), atol=1e-7)


def test_norms_by_hand():
    z, r = oracle.norm_rows(np.array([[1.0, 3.0]]), "layer", 0.0)
    assert np.allclose(z, [[-1.0, 1.0]]) and np.allclose(r, 1.0)
    z, r = oracle.norm_rows(np.array([[3.0, 4.0]]), "rms", 0.0)
    assert np.allclose(z, np.array([[3.0, 4.0]]) / math.sqrt(12.5))
    y = _rand(1, 2, 3, 4, 8)
    assert np.allclose(oracle.norm_gate(y, None, "layer", 1e-5), oracle.group_norm(y, 1e-5))
    g = _rand(2, 2, 3, 4, 8)
    assert np.allclose(oracle.norm_gate(y, g, "layer", 1e-5),
                       oracle.gated(oracle.group_norm(y, 1e-5), g))
    assert np.allclose(oracle.norm_gate(y, g.swapaxes(1, 2), "layer", 1e-5, True),
                       oracle.gated(oracle.group_norm(y, 1e-5), g).swapaxes(1, 2))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("token_major", [False, True])
def test_norm_gate_backward_against_differences(kind, token_major):
    y, g = _rand(1, 1, 2, 3, 8), _rand(2, *((1, 3, 2, 8) if token_major else (1, 2, 3, 8)))
    d_o = _rand(3, *g.shape)
    loss = lambda: (oracle.norm_gate(y, g, kind, 1e-3, token_major) * d_o).sum()  # noqa: E731
    dy, dg = oracle.norm_gate_backward(y, g, d_o, kind, 1e-3, token_major)
    assert np.allclose(dy, _difference(loss, y), atol=1e-7)
    assert np.allclose(dg, _difference(loss, g), atol=1e-7)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_add_norm_backward_against_differences(post, pre):
    x, res, w, wp = _rand(1, 4, 6), _rand(2, 4, 6), _rand(3, 6), _rand(4, 6)
    d_y, d_r = _rand(5, 4, 6), _rand(6, 4, 6)
    args = (post, pre, 1.5, 0.7, 1e-3)

    def loss():
        r, y = oracle.add_norm(x, res, w, wp, *args)
        return (y * d_y).sum() + (r * d_r).sum()

    r, _ = oracle.add_norm(x, res, w, wp, *args)
    got = oracle.add_norm_backward(x, r, w, d_y, d_r, wp, *args)
    for g, wrt in zip(got, (x, res, w, wp)):
        assert np.allclose(g, _difference(loss, wrt), atol=1e-7)
